"""The feed-forward operators' host side on the CPU: exports, argument checks
and the work split (no GPU)."""
import ctypes
import itertools

import pytest
import torch

import mixed_precision_dense_sm_gb300 as lib

F16, BF16, F32 = lib.GEMM_F16, lib.GEMM_BF16, lib.GEMM_F32


def test_declared():
    names = lib.declared_symbols()
    for n in ("glu_forward", "glu_backward", "glu_plan_query", "norm_block_forward",
              "norm_block_backward", "norm_block_backward_workspace", "grad_clip", "grad_clip_workspace"):
        assert n in names and hasattr(lib.lib, n)


def plan(M=64, F=512, K=256, X=256, ldx=None, W=256, ldw=None, H=256, ldh=None, dt=(BF16, BF16, BF16), **kw):
    return lib.glu_plan_query(M, F, K, X, ldx or max(K, 1), W, ldw or max(K, 1), H, ldh or max(F, 1), dt, **kw)


def test_glu_arguments():
    assert plan()[0] == 0
    assert plan(P=256, ldp=1024)[0] == 0 and plan(bias=4, act=lib.ACT_SILU)[0] == 0
    for bad in (dict(M=-1), dict(F=-1), dict(K=-1), dict(F=2 ** 30), dict(ldx=255), dict(ldw=255),
                dict(ldh=511), dict(X=0), dict(W=0), dict(H=0), dict(X=257), dict(H=257),
                dict(dt=(BF16, F16, BF16)), dict(dt=(BF16, BF16, 7)), dict(act=9), dict(act=-1),
                dict(bias=256, bias_dtype=5), dict(bias=258, bias_dtype=F32), dict(P=256, ldp=1023),
                dict(P=257, ldp=1024)):
        assert plan(**bad)[0] == 1, bad
    assert plan(dt=(F32, F32, F32))[0] == 2
    assert lib.glu_forward(None, 1, 1, 1, 256, 1, 256, 1, 256, 1, (BF16, BF16, BF16)) == 1
    assert lib.glu_backward(None, 1, 1, 1, 256, 1, 256, 2, 256, 1, 256, 1, BF16, 256, 2) == 1


@pytest.mark.parametrize("seed", range(6))
def test_glu_plans_cover_the_problem(seed):
    """Invariants of the plan on random problems: every output tile and K block
    is there once, the kernels' widths, and a split in K only where allowed."""
    import random
    rng = random.Random(seed)
    for _ in range(300):
        M, F, K = (int(2 ** rng.uniform(0, b)) for b in (13.5, 14.5, 13.5))
        ld = K + rng.choice([0, 0, 1, 8])
        st, p = plan(M=M, F=F, K=K, ldx=ld, ldw=K + rng.choice([0, 0, 1, 8]),
                     ldh=F + rng.choice([0, 3, 8]), dt=(BF16, BF16, rng.choice([BF16, F16, F32])))
        assert st == 0
        if p["path_name"] == "dot":
            assert M <= 2 and K % 8 == 0
            continue
        pad = p["pack_a"] and p["pack_b"]
        kk = -(-K // 128) * 128 if pad else K
        assert p["k_blocks"] == -(-kk // p["block_k"])
        if p["swap_ab"]:
            assert M <= 128 and p["tiles_m"] == -(-F // 64) and p["block_n"] * p["tiles_n"] >= M
        else:
            assert p["block_m"] * p["tiles_m"] >= M and p["block_n"] // 2 * p["tiles_n"] >= F
            assert p["block_m"] * (p["tiles_m"] - 1) < M and p["block_n"] // 2 * (p["tiles_n"] - 1) < F
        assert p["num_tiles"] == p["tiles_m"] * p["tiles_n"]
        if p["path_name"] == "skinny" and p["sk_len"] == 0 and p["split_k"] > 1:
            assert p["grid"] == p["num_tiles"] * p["split_k"] and p["split_k"] in (2, 4, 8)
            assert p["block_n"] >= 4 * p["split_k"] and p["k_blocks"] >= 2 * p["split_k"]
        if p["sk_len"]:
            cg = 2 if p["path_name"] == "tiled_2sm" else 1
            assert p["grid"] // cg * p["sk_len"] >= p["num_tiles"] * p["k_blocks"]


def norm(M=4, N=64, X=256, Z=256, XO=256, Y=256, x=F32, z=BF16, ld=64, **kw):
    b = dict(pre=1, post=1, pre_weight=None, pre_bias=None, post_weight=None, post_bias=None, gate=None,
             ld_gate=64, gate_rows=1, vec_dtype=F32, scale=1.0, eps=1e-5)
    b.update(kw)
    return lib.norm_block_forward(M, N, X, ld, Z, ld, XO, ld, Y, ld, x, z, lib.NormBlock(**b))


def test_norm_arguments():
    inf, nan = float("inf"), float("nan")
    for bad in (dict(M=-1), dict(N=-1), dict(M=2 ** 31), dict(X=0), dict(X=258), dict(Z=257), dict(Y=257),
                dict(XO=0), dict(Z=0), dict(Z=0, XO=0, Y=0), dict(ld=63), dict(x=5), dict(z=-1),
                dict(pre=3), dict(post=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=inf), dict(eps=nan),
                dict(scale=inf), dict(scale=nan), dict(pre_weight=256, vec_dtype=3),
                dict(post_bias=258), dict(gate=256, gate_rows=0), dict(gate=256, ld_gate=63)):
        assert norm(**bad) == 1, bad
    assert norm(x=BF16, z=F32) == 2 and norm(x=BF16, z=F16) == 2
    assert norm(N=lib.NORM_MAX_N + 1, ld=lib.NORM_MAX_N + 1) == 2
    assert norm(M=0) == 0 and norm(N=0, X=0, Z=256, XO=256, Y=0) == 0


def back(M=4, N=64, XO=256, Z=256, dY=256, dXO=256, dX=256, dZ=256, x=F32, z=BF16, ws=256, nbytes=0,
         grads=None, **kw):
    b = dict(pre=1, post=1, gate=None, ld_gate=64, gate_rows=1, vec_dtype=F32, scale=1.0, eps=1e-5)
    b.update(kw)
    g = dict(d_pre_weight=None, d_pre_bias=None, d_post_weight=None, d_post_bias=None, d_gate=None,
             grad_dtype=F32)
    g.update(grads or {})
    return lib.norm_block_backward_raw(M, N, XO, N, Z, N, dY, N, dXO, N, dX, N, dZ, N, x, z,
                                       lib.NormBlock(**b), lib.NormBlockGrads(**g), ws, nbytes)


def test_norm_backward_arguments():
    for bad in (dict(XO=0), dict(XO=258), dict(dY=257), dict(dXO=258), dict(dX=258), dict(dZ=257),
                dict(Z=0), dict(Z=0, dZ=0, grads=dict(d_post_weight=256)),
                dict(grads=dict(d_gate=256)), dict(grads=dict(d_pre_weight=258)),
                dict(grads=dict(d_pre_weight=256, grad_dtype=4)), dict(grads=dict(d_pre_weight=256), ws=0),
                dict(grads=dict(d_pre_weight=256), ws=264)):
        assert back(**bad) == 1, bad


def test_norm_workspace():
    w = lib.norm_block_backward_workspace
    for bad in ((-1, 8, 1, 152), (8, -1, 1, 152), (8, 8, 0, 152), (8, 8, 1, -1)):
        assert w(*bad) == -1
    for M, N, rows, sms in itertools.product((0, 1, 5, 303, 304, 305, 8192, 100000), (1, 4096), (1, 2, 3, 100, 8192),
                                             (1, 16, 152)):
        b = w(M, N, rows, sms)
        lines = b // (16 * N) - 16                  # (16 more for the second step of the sums)
        assert b == (lines + 16) * 16 * N and lines >= 1
        # no more lines than rows or twice the SMs, but one for every gate group
        groups = -(-max(M, 1) // rows) if 1 < rows < M else 1
        assert lines <= max(M, 1) + groups and lines <= 2 * sms + 2 * groups


def clip(grads=(256,), outs=None, sizes=(4,), dtypes=(F32,), max_norm=1.0, inv_scale=1.0, norm=256, ws=256,
         nbytes=1 << 20):
    return lib.grad_clip_raw(list(grads), None if outs is None else list(outs), list(sizes), list(dtypes),
                             max_norm, inv_scale, norm, ws, nbytes)


def test_clip_arguments():
    inf, nan = float("inf"), float("nan")
    for bad in (dict(grads=(0,)), dict(grads=(257,), dtypes=(BF16,)), dict(grads=(258,)), dict(outs=(0,)),
                dict(outs=(258,)), dict(sizes=(-1,)), dict(dtypes=(3,)), dict(max_norm=0.0),
                dict(max_norm=-1.0), dict(max_norm=nan), dict(inv_scale=0.0), dict(inv_scale=inf),
                dict(inv_scale=nan), dict(norm=0), dict(norm=258), dict(ws=0), dict(ws=264),
                dict(grads=(256, 256), sizes=(4, 4), dtypes=(F32, F32)),
                dict(grads=(256, 512), outs=(256, 512), sizes=(4, -4), dtypes=(F32, F32))):
        assert clip(**bad) == 1, bad
    # outputs that meet each other or another gradient
    f = dict(sizes=(4, 4), dtypes=(F32, F32))
    for g, o in (((256, 512), (1024, 1036)), ((256, 512), (512, 1024)), ((256, 512), (1024, 264)),
                 ((256, 264), (256, 264)), ((256, 256), (1024, 1024)), ((256, 512), (260, 1024))):
        assert clip(grads=g, outs=o, **f) == 1, (g, o)
    assert lib.lib.grad_clip(1, None, None, None, None, 1.0, 1.0, 256, 256, 1 << 20, None) == 1
    assert lib.lib.grad_clip(-1, None, None, None, None, 1.0, 1.0, 256, 256, 1 << 20, None) == 1
    assert lib.grad_clip_workspace(-1, 152) == -1 and lib.grad_clip_workspace(1, -1) == -1
    assert lib.grad_clip_workspace(0, 152) == lib.grad_clip_workspace(512, 152)
    assert lib.grad_clip_workspace(513, 152) == 2 * lib.grad_clip_workspace(1, 152)


def test_tensors_must_be_on_the_gpu():
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (lambda: lib.norm_block(t), lambda: lib.norm_block_backward(t, t), lambda: lib.grad_clip([t], 1.0)):
        with pytest.raises(ValueError):
            f()


def test_struct_layouts():
    """The ctypes structures are laid out as the C ones (size checked by natural alignment)."""
    assert ctypes.sizeof(lib.GluForward) == 40 and ctypes.sizeof(lib.GluBackward) == 88
    assert ctypes.sizeof(lib.NormBlock) == 80 and ctypes.sizeof(lib.NormBlockGrads) == 48


@pytest.mark.parametrize("shape,stride,ld", [((4, 1), (0, 1), 0), ((4, 1), (0, 0), 0), ((4, 1), (3, 7), 3),
                                             ((4, 8), (0, 1), 0), ((4, 8), (2, 1), 2), ((1, 8), (0, 1), 8),
                                             ((1, 8), (99, 1), 8), ((1, 1), (0, 0), 1), ((4, 0), (0, 1), 1),
                                             ((0, 8), (0, 1), 8), ((4, 8), (12, 1), 12)])
def test_row_pitch_of_a_view(shape, stride, ld):
    """Broadcast and overlapping rows keep a pitch below the row length, which
    the library refuses."""
    t = torch.empty(64).as_strided(shape, stride)
    assert lib._mat(t, "t", *shape, torch.float32, -1) == (t.data_ptr(), ld)
    if ld < max(shape[1], 1):
        assert plan(M=shape[0], K=shape[1], ldx=ld or -1)[0] == 1


@pytest.mark.parametrize("c,es", [(lib.GEMM_F32, 4), (BF16, 2), (lib.GEMM_F16, 2)])
def test_tma_stores_need_rows_of_whole_pieces(c, es):
    """A TMA store clips by 16 bytes: only rows of whole 16-byte pieces take it,
    whatever the pitch (of C, and of the gated layer's H)."""
    seen = set()
    for N in range(2384, 2401):
        want = int(N * es % 16 == 0)
        st, p = lib.gemm_plan_query("N", "T", 20000, N, 2048, 1.0, 256, 2048, 256, 2048, 0.0, 256, 2400,
                                    (BF16, BF16, c))
        assert st == 0 and p["c_tma"] == want, (N, p)
        st, p = plan(M=20000, F=N, K=2048, ldh=2400, dt=(BF16, BF16, c))
        assert st == 0 and p["c_tma"] == want, (N, p)
        seen.add(want)
    assert seen == {0, 1}
