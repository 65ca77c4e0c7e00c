"""The operators that prepare and verify drafted tokens: qkv_norm_rope_fp4, kv_dequant_fp4 and
tree_attn_decode against plain formulas in 64 bits, their refusals, and a run of them together.

Tolerances:
* the KV row's bf16 value, cache bytes and read-back values: exact;
* queries: half a bf16 step of the value (2^-8 relative) and, before it, fp32 arithmetic: a sum of
  squares of at most 1024 terms, at most 32 of them in sequence per lane and 5 joining steps, so
  r is off by at most 20 x 2^-24 relative and a rotated channel by a few 2^-24 of |u_a| + |u_b|:
  2^-18 (|u_a| + |u_b|) r covers both;
* tree attention: half a bf16 step of the value; the probabilities are multiplied as fp16 (2^-11
  relative each), and a logit is an fp32 sum of 512 products, whose order and rounding leave at
  most 2^-16 of scale x sum |q v|. With A = sum_j p_j |v_j| an output is off by at most
  2^-8 |o| + (2^-11 + 2 dz) A, lse by dz and its own fp32 rounding. No floating type holds every
  probability to a relative 2^-11: fp16 has a step of 2^-24 below 2^-14, so a p that is stored as at
  least 2^3 at the row's maximum is off by up to 2^-25 / 2^3 = 2^-28 of that maximum (<= 1), which
  adds 2^-28 sum_j |v_j|.
  (A probability goes as two fp16 by now and is nearer than that; test_tree_rows_that_cancel counts it.)
"""
import ctypes

import numpy as np
import pytest
import torch

import synth
from fp4_sparse_attention_kv_b200 import binding
from oracle import fp4kv_oracle as O
from tests import parity as P

DEV = "cuda"
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def fk(cuda_lib):
    import fp4_sparse_attention_kv_b200 as fk
    return fk


# ----------------------------------------------------------------------------------------
# plain forms, 64 bits
# ----------------------------------------------------------------------------------------

def plain_norm_rope(x, w, pos, table, rope, half, eps):
    """x bf16 [..., d] with one position per leading row -> (y, |u_a| + |u_b| (or |u|) times r), fp64."""
    x = x.double()
    d = x.shape[-1]
    r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / d + eps)
    u = x * w.double() if w is not None else x.clone()
    y, mag = u.clone(), u.abs()
    if rope:
        t = table.double()[pos]
        c, s = t[:, : rope // 2], t[:, rope // 2:]
        if x.dim() == 3:
            c, s = c[:, None], s[:, None]
        z = torch.arange(d - rope, d, device=x.device)
        ia, ib = (z[: rope // 2], z[rope // 2:]) if half else (z[0::2], z[1::2])
        a, b = u[..., ia], u[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y * r, mag * r


def bf16_of_f64(y):
    """The nearest fp32 value, rounded to bf16."""
    return y.float().bfloat16()


def cache_values(packed, scales):
    return torch.from_numpy(O.kv_dequant_fp4(packed.cpu().numpy(), scales.cpu().numpy()))


def plain_tree(q, packed, scales, lens, mask, drafts, idx, scale, b, t):
    """One token's (out [H, 512], lse [H], bound on what out may be off before its rounding, dz [H]), fp64."""
    cap = packed.shape[0]
    n = max(0, min(int(lens[b]), cap))
    pre = list(range(n)) if idx is None else [int(i) for i in idx[b].tolist() if 0 <= i < n]
    m = int(mask[b, t])
    rows = pre + [n + j for j in range(drafts[b]) if (m >> j) & 1 and n + j < cap]
    H = q.shape[2]
    if not rows:
        z = torch.zeros(H, 512, dtype=torch.float64)
        return z, torch.full((H,), -np.inf, dtype=torch.float64), z, torch.zeros(H, dtype=torch.float64)
    r = torch.tensor(rows, device=packed.device)
    v = cache_values(packed[r], scales[r])
    qq = q[b, t].double().cpu()
    z = qq @ v.T * scale
    p = torch.softmax(z, -1)
    dz = 2.0 ** -16 * abs(scale) * (qq.abs() @ v.abs().T).amax(-1)
    return p @ v, torch.logsumexp(z, -1), p @ v.abs() * (2.0 ** -11 + 2 * dz[:, None]) + 2.0 ** -28 * v.abs().sum(0), dz


def check_tree(fk, q, packed, scales, lens, mask, drafts, idx, scale, out, lse, what=""):
    B, T = q.shape[:2]
    for b in range(B):
        for t in range(drafts[b]):
            ro, rl, slack, dz = plain_tree(q, packed[b], scales[b], lens, mask, drafts, idx, scale, b, t)
            o, l = out[b, t].double().cpu(), lse[b, t].double().cpu()
            assert torch.isfinite(o).all(), f"{what} b={b} t={t}: out not finite"
            tol = 2.0 ** -8 * ro.abs() + slack
            bad = ((o - ro).abs() - tol).max()
            assert bad <= 0, f"{what} b={b} t={t}: out off by {bad:.3e} above its tolerance"
            inf = torch.isinf(rl)
            assert torch.equal(torch.isneginf(l), inf), f"{what} b={b} t={t}: lse -inf"
            if not inf.any():
                assert ((l - rl).abs() <= dz + 2.0 ** -21 * rl.abs() + 2.0 ** -20).all(), f"{what} b={b} t={t}: lse"


def table_of(top, rope, seed=0):
    f = 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64) / max(rope, 1))
    a = torch.arange(top, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().to(DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make_cache(fk, B, cap, seed, d=512):
    x = torch.randn(B * cap, d, generator=gen(seed), device=DEV)
    x[:, ::101] *= 20.0
    packed = torch.empty(B, cap, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(B, cap, d // 16, dtype=torch.uint8, device=DEV)
    fk.kv_quant_fp4(x.bfloat16(), packed.view(-1, d // 2), scales.view(-1, d // 16))
    return packed, scales


def tree_masks(B, T, seed):
    """Random trees: every token sees itself and its ancestors."""
    rng = np.random.default_rng(seed)
    m = np.zeros((B, T), dtype=np.uint64)
    for b in range(B):
        for j in range(T):
            par = int(rng.integers(-1, j)) if j else -1
            m[b, j] = (m[b, par] if par >= 0 else np.uint64(0)) | np.uint64(1 << j)
    return torch.from_numpy(m.view(np.int64)).to(DEV)


# ----------------------------------------------------------------------------------------
# refusals (CPU): the C entries check before the first CUDA call, the binding before that
# ----------------------------------------------------------------------------------------

def _c(name, *args):
    L = binding.lib()
    return getattr(L, name)(*args), L.fp4kv_last_error().decode()


FAKE = 0x10000


def _norm_args(**k):
    a = dict(q=FAKE, qts=64 * 512, qhs=512, H=64, qw=None, qo=FAKE, kv=FAKE, kvs=512, kw=None, kvo=None, dst=None,
             packed=FAKE, scales=FAKE, cap=16, n=4, d=512, rope=64, half=0, pos=FAKE, cs=FAKE, mp=10, eps=1e-6, st=None)
    a.update(k)
    return list(a.values())


@pytest.mark.parametrize("change, status, word", [
    (dict(d=48), 2, "d=48"), (dict(d=1056, kvs=1056), 2, "d=1056"), (dict(rope=24), 2, "rope_dim=24"),
    (dict(rope=528), 2, "rope_dim=528"), (dict(d=1024, kvs=1024, qhs=1024, rope=528), 2, "rope_dim=528"), (dict(rope=-16), 2, "rope_dim"), (dict(eps=0.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"), (dict(eps=float("inf")), 1, "eps"), (dict(q=None, kv=None), 1, "null q and kv"),
    (dict(H=0), 2, "H=0"), (dict(H=129), 2, "H=129"), (dict(qo=None), 1, "q_out"), (dict(packed=None), 1, "neither"),
    (dict(scales=None), 1, "scales"), (dict(pos=None), 1, "positions"), (dict(cs=None), 1, "cos_sin"),
    (dict(qhs=504), 1, "strides"), (dict(qts=516), 1, "strides"), (dict(kvs=516), 1, "kv_row_stride"),
    (dict(kvs=0), 1, "kv_row_stride"), (dict(q=FAKE + 8), 1, "aligned"), (dict(kv=FAKE + 2), 1, "aligned"),
    (dict(cs=FAKE + 4), 1, "aligned"), (dict(packed=FAKE + 4), 1, "aligned"), (dict(n=17), 1, "cap_rows"),
    (dict(n=-1), 1, "negative"), (dict(mp=-1), 1, "negative"), (dict(kv=None), 1, "packed needs kv"),
])
def test_norm_rope_refusals(change, status, word):
    st, msg = _c("fp4kv_qkv_norm_rope_fp4", *_norm_args(**change))
    assert st == status and word in msg, (st, msg)


def test_no_rows_is_a_success_without_pointers():
    st, msg = _c("fp4kv_qkv_norm_rope_fp4", *_norm_args(n=0, qo=None, packed=None, scales=None, pos=None, cs=None))
    assert (st, msg) == (0, "")
    assert _c("fp4kv_kv_dequant_fp4", None, None, 0, 512, None, 0, None, 0, 512, None) == (0, "")


@pytest.mark.parametrize("change, status, word", [
    (dict(d=40), 2, "d=40"), (dict(packed=None), 1, "null"), (dict(scales=None), 1, "null"), (dict(out=None), 1, "null"),
    (dict(stride=504), 1, "stride"), (dict(stride=516), 1, "stride"), (dict(out=FAKE + 8), 1, "aligned"),
    (dict(packed=FAKE + 8), 1, "aligned"), (dict(n=11), 1, "cap_rows"), (dict(n=-1), 1, "negative"),
    (dict(cap=-1), 1, "negative"),
])
def test_dequant_refusals(change, status, word):
    a = dict(packed=FAKE, scales=FAKE, cap=10, d=512, src=None, n=4, out=FAKE, f32=0, stride=512, st=None)
    a.update(change)
    st, msg = _c("fp4kv_kv_dequant_fp4", *a.values())
    assert st == status and word in msg, (st, msg)


@pytest.mark.parametrize("change, status, word", [
    (dict(B=0), 2, "B=0"), (dict(B=65536), 2, "B=65536"), (dict(T=0), 2, "T=0"), (dict(T=65), 2, "T=65"),
    (dict(H=0), 2, "H=0"), (dict(H=129), 2, "H=129"), (dict(d=256), 2, "d=256"), (dict(top_k=0), 2, "top_k=0"),
    (dict(top_k=(1 << 20) + 1), 2, "top_k"), (dict(idx=None), 2, "top_k"), (dict(cap=0), 2, "cap=0"),
    (dict(cap=1 << 31), 2, "cap"), (dict(q=None), 1, "null"), (dict(mask=None), 1, "null"), (dict(ws=None), 1, "null"),
    (dict(out=FAKE + 8), 1, "misaligned"), (dict(ws=FAKE + 16), 1, "misaligned"), (dict(mask=FAKE + 4), 1, "misaligned"),
    (dict(wsb=255), 4, "ws_bytes"), (dict(B=65535, T=64, H=128, idx=None, top_k=0, cap=(1 << 31) - 8), 2, "tiles"),
])
def test_tree_refusals(change, status, word):
    a = dict(q=FAKE, B=2, T=5, H=64, d=512, packed=FAKE, scales=FAKE, cap=100, lens=FAKE, nd=None, mask=FAKE, idx=FAKE,
             top_k=16, scale=1.0, out=FAKE, lse=None, ws=FAKE, wsb=1 << 30, st=None)
    a.update(change)
    a["scale"] = ctypes.c_float(a["scale"])
    st, msg = _c("fp4kv_tree_attn_decode", *a.values())
    assert st == status and word in msg, (st, msg)


def test_tree_workspace_sizes():
    wb = binding.workspace_bytes
    assert wb(binding.OP_TREE_ATTN, 4, 32784, 16 * 64, 0) >= 256
    assert wb(binding.OP_TREE_ATTN, 4, 32784, 0, 0) == 0
    # the smaller problem never needs more
    assert wb(binding.OP_TREE_ATTN, 1, 100, 8, 0) <= wb(binding.OP_TREE_ATTN, 1, 100000, 8 * 64, 0)


@pytest.mark.parametrize("cap, top_k", [(100, 0), (512, 0), (600, 0), (1000, 0), (1300, 0), (70000, 0), (70000, 512), (70000, 800)])
def test_a_tree_workspace_for_a_batch_serves_every_smaller_one(cap, top_k):
    sizes = [binding.workspace_bytes(binding.OP_TREE_ATTN, B, cap, rows, top_k) for rows in (8, 128, 500) for B in range(1, 160)]
    for at in range(0, len(sizes), 159):
        assert sizes[at:at + 159] == sorted(sizes[at:at + 159])


@pytest.mark.parametrize("shape", [(2, 0), (0, 0), (2,), (2, 1, 4)])
def test_binding_refuses_a_selection_without_entries(shape):
    """Its address is null, the library's word for "every row"."""
    idx = torch.empty(shape, dtype=torch.int32)
    assert idx.numel() or idx.data_ptr() == 0
    with pytest.raises(ValueError, match="idx"):
        binding.tree_attn_decode(torch.zeros(2, 1, 1, 512, dtype=torch.bfloat16), None, None, None, None, idx=idx)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf"), 1e39])
def test_tree_refuses_a_scale_that_is_not_finite(scale):
    """A NaN scale gave every token the mean of what it sees."""
    args = [FAKE, 2, 5, 64, 512, FAKE, FAKE, 100, FAKE, None, FAKE, None, 0, ctypes.c_float(scale), FAKE, None, FAKE, 1 << 30, None]
    st, msg = _c("fp4kv_tree_attn_decode", *args)
    assert st == 1 and "sm_scale" in msg, (st, msg)


@gpu
def test_tree_a_selection_of_nothing(fk):
    """Refused without a column, the drafts alone with one column of -1."""
    B, T, H, n = 2, 3, 10, 200
    packed, scales = make_cache(fk, B, n + T, 150)
    q = torch.randn(B, T, H, 512, generator=gen(151), device=DEV).bfloat16()
    lens, mask = torch.tensor([n, 77], dtype=torch.int32, device=DEV), tree_masks(B, T, 2)
    with pytest.raises(ValueError, match="idx"):
        fk.tree_attn_decode(q, packed, scales, lens, mask, idx=torch.empty(B, 0, dtype=torch.int32, device=DEV))
    run_tree(fk, B, T, H, [n, 77], None, n + T, idx=torch.full((B, 1), -1, dtype=torch.int32, device=DEV), q=q, mask=mask,
             cache=(packed, scales))


def test_binding_refuses_cpu_tensors_and_missing_arguments():
    x = torch.zeros(2, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.qkv_norm_rope_fp4(None, None)
    with pytest.raises(TypeError):
        binding.qkv_norm_rope_fp4(None, x)
    with pytest.raises(TypeError):
        binding.kv_dequant_fp4(torch.zeros(2, 256, dtype=torch.uint8), torch.zeros(2, 32, dtype=torch.uint8))
    with pytest.raises(TypeError):
        binding.tree_attn_decode(torch.zeros(1, 1, 1, 512, dtype=torch.bfloat16), None, None, None, None)


# ----------------------------------------------------------------------------------------
# kv_dequant_fp4
# ----------------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequant_every_code_and_scale(fk, dtype):
    """All 256 code bytes under all 254 finite scale bytes."""
    sc = torch.tensor([s for s in range(256) if s & 0x7f != 0x7f], dtype=torch.uint8)
    packed = torch.arange(256, dtype=torch.uint8).view(1, 256).repeat(len(sc), 1).to(DEV)
    scales = sc[:, None].repeat(1, 32).to(DEV)
    got = fk.kv_dequant_fp4(packed, scales, dtype=dtype)
    want = cache_values(packed, scales)
    assert torch.equal(got.double().cpu(), want)
    assert torch.equal(torch.signbit(got.cpu()), torch.signbit(want))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d, cap, n", [(32, 5, 3), (64, 1, 1), (96, 700, 1001), (128, 33, 4000), (512, 1000, 257),
                                       (512, 3000, 60001), (576, 64, 129), (1024, 100, 3001)])
def test_dequant_gather(fk, d, cap, n, dtype):
    packed, scales = make_cache(fk, 1, cap, d + n, d)
    packed, scales = packed[0], scales[0]
    src = torch.randint(0, cap, (n,), generator=gen(n), device=DEV)
    src[::7] = torch.tensor([-1, cap, 1 << 40, -(1 << 40)], device=DEV).repeat(n)[: len(src[::7])]
    wide = torch.full((n, d + 8), 7.0, dtype=dtype, device=DEV)  # a row stride above d
    got = fk.kv_dequant_fp4(packed, scales, src_row=src, out=wide[:, :d])
    ok = (src >= 0) & (src < cap)
    want = cache_values(packed, scales).to(DEV)[src.clamp(0, cap - 1)] * ok[:, None]
    assert torch.equal(got.double(), want)
    assert (wide[:, d:] == 7.0).all()
    assert torch.equal(fk.kv_dequant_fp4(packed, scales, dtype=dtype).double().cpu(), cache_values(packed, scales))


@gpu
def test_dequant_inverts_the_quantizer_and_takes_no_rows(fk):
    packed, scales = make_cache(fk, 2, 40, 3)
    x = fk.kv_dequant_fp4(packed, scales)
    p2, s2 = torch.empty_like(packed), torch.empty_like(scales)
    fk.kv_quant_fp4(x, p2.view(-1, 256), s2.view(-1, 32))
    assert torch.equal(fk.kv_dequant_fp4(p2, s2), x)  # every group has a code 6, so its scale comes back too
    none = fk.kv_dequant_fp4(packed, scales, src_row=torch.empty(0, dtype=torch.int64, device=DEV))
    assert none.shape == (0, 512)
    with pytest.raises(ValueError):
        fk.kv_dequant_fp4(packed, scales, out=torch.empty(79, 512, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        fk.kv_dequant_fp4(packed, scales, out=torch.empty(80, 512, dtype=torch.float16, device=DEV))


# ----------------------------------------------------------------------------------------
# qkv_norm_rope_fp4
# ----------------------------------------------------------------------------------------

def norm_inputs(n, H, d, seed, loud=True):
    g = gen(seed)
    q = (torch.randn(n, max(H, 1), d, generator=g, device=DEV) * 3).bfloat16() if H else None
    kv = torch.randn(n, d, generator=g, device=DEV)
    if loud and n:
        kv[:, 3] *= 50.0
        kv[0] = 0.0  # a row of zeros
        kv[-1] *= 1e-3
    qw = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16()
    kw = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16()
    return q, kv.bfloat16(), qw, kw


def check_q(got, q, w, pos, table, rope, half, eps):
    y, mag = plain_norm_rope(q, w, pos, table, rope, half, eps)
    tol = 2.0 ** -8 * y.abs() + 2.0 ** -18 * mag
    assert ((got.double() - y).abs() <= tol).all()


@gpu
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("n, H, d, rope, half", [
    (1, 64, 512, 64, False), (1, 1, 32, 0, False), (3, 1, 32, 32, True), (130, 5, 64, 64, False), (777, 32, 128, 64, True),
    (33, 12, 96, 48, False), (33, 12, 96, 96, True), (50, 8, 192, 128, True), (64, 3, 256, 16, False),
    (64, 128, 320, 0, False), (500, 2, 512, 512, True), (129, 16, 576, 64, False), (17, 7, 1024, 128, True), (40, 3, 1024, 512, True),
    (20000, 0, 1024, 112, True), (40000, 0, 128, 48, True), (40000, 0, 192, 96, False), (30000, 0, 64, 0, False), (20000, 0, 512, 16, True),
    (5000, 0, 512, 64, True), (60000, 0, 512, 64, False)])
def test_norm_rope(fk, n, H, d, rope, half, weight):
    q, kv, qw, kw = norm_inputs(n, H, d, n + d)
    qw, kw = (qw, kw) if weight else (None, None)
    top = 4096
    table = table_of(top, rope)
    pos = torch.randint(0, top, (n,), generator=gen(n), device=DEV)
    cap = n + 9
    dst = torch.randperm(cap, generator=gen(d), device=DEV)[:n]
    skip = torch.arange(n, device=DEV) % 11 == 5
    dst = torch.where(skip, torch.where(torch.arange(n, device=DEV) % 2 == 0, -1, cap), dst)
    packed = torch.full((cap, d // 2), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((cap, d // 16), 0xCD, dtype=torch.uint8, device=DEV)
    kv_out = torch.full((n, d), 7.0, dtype=torch.bfloat16, device=DEV)
    for eps in (1e-6, 1e-2):
        qo, ko = fk.qkv_norm_rope_fp4(q, kv, positions=pos, cos_sin=table, rope_dim=rope, rope_half=half, q_weight=qw,
                                      kv_weight=kw, eps=eps, packed=packed, scales=scales, dst_row=dst, kv_out=kv_out)
        if H:
            check_q(qo, q, qw, pos, table, rope, half, eps)
        want = bf16_of_f64(plain_norm_rope(kv, kw, pos, table, rope, half, eps)[0])
        assert torch.equal(ko, want)
        op, os_ = O.kv_quant_fp4(P.to_f64(want))
        live = (dst >= 0) & (dst < cap)
        assert torch.equal(packed[dst[live]].cpu(), torch.from_numpy(op)[live.cpu()])
        assert torch.equal(scales[dst[live]].cpu(), torch.from_numpy(os_)[live.cpu()])
        rest = torch.ones(cap, dtype=torch.bool, device=DEV)
        rest[dst[live]] = False
        assert (packed[rest] == 0xAB).all() and (scales[rest] == 0xCD).all()


@gpu
@pytest.mark.parametrize("n, d", [(5, 128), (70000, 128), (9, 512), (20000, 512), (6, 1024)])
def test_norm_rope_rows_that_are_not_finite(fk, n, d):
    """By the formula a NaN channel makes its row NaN, and an infinite one (r = 0) zeros with NaN in its
    own place (and, rotated, in its partner's). The cache holds what kv_quant_fp4 makes of that."""
    rope = 32
    x = torch.randn(n, d, generator=gen(71), device=DEV).bfloat16()
    x[0, 3] = float("nan")
    x[1, 0] = float("inf")
    x[2, d - 1] = float("-inf")     # rotated with channel d - 2
    x[n - 1, d - rope] = float("nan")
    x[n - 2, d // 2] = 3.3e38       # finite
    table = table_of(64, rope)
    pos = torch.arange(n, device=DEV) % 64
    packed, scales = (torch.zeros(n, d // k, dtype=torch.uint8, device=DEV) for k in (2, 16))
    q, kv = fk.qkv_norm_rope_fp4(None, x, positions=pos, cos_sin=table, rope_dim=rope, packed=packed, scales=scales,
                                 kv_out=torch.empty_like(x))
    p2, s2 = torch.zeros_like(packed), torch.zeros_like(scales)
    fk.kv_quant_fp4(kv, p2, s2)
    assert torch.equal(packed, p2) and torch.equal(scales, s2)
    want = bf16_of_f64(plain_norm_rope(x, None, pos, table, rope, False, 1e-6)[0])
    assert torch.isnan(kv[0]).all() and torch.isnan(kv[n - 1]).all()
    for r, places in ((1, [0]), (2, [d - 2, d - 1])):
        nan = torch.zeros(d, dtype=torch.bool, device=DEV)
        nan[places] = True
        assert torch.isnan(kv[r][nan]).all() and (kv[r][~nan] == 0).all()
    rest = torch.isfinite(x).all(1)
    assert torch.equal(kv[rest].float(), want[rest].float())


@gpu
@pytest.mark.parametrize("rope, half", [(0, False), (64, False), (64, True)])
@pytest.mark.parametrize("n, H, d", [(3, 5, 512), (700, 64, 512), (40, 7, 128), (20, 9, 1024)])
def test_norm_rope_queries_that_are_not_finite(fk, n, H, d, rope, half):
    """By the formula, as for KV rows: NaN makes its head NaN; an infinity makes r 0, so NaN in its own place (and,
    rotated, in its partner's) and zeros elsewhere. The other heads are as without."""
    q = torch.randn(n, H, d, generator=gen(75), device=DEV).bfloat16()
    w = (1 + 0.2 * torch.randn(d, generator=gen(76), device=DEV)).bfloat16()
    table, pos = (table_of(64, rope), torch.arange(n, device=DEV) % 64) if rope else (None, None)
    x = q.clone()
    x[0, 0, 3] = float("nan")
    x[0, 1, 0] = float("inf")         # (its neighbour is not rotated with it)
    x[1, 2, d - 65] = float("-inf")
    x[n - 1, H - 1, 17] = float("inf")
    x[2, 0, d - 1] = float("-inf")    # rotated, if any is, with channel d - 2, or d - 1 - rope / 2
    how = dict(positions=pos, cos_sin=table, rope_dim=rope, rope_half=half, q_weight=w)
    want, got = fk.qkv_norm_rope_fp4(q, None, **how)[0], fk.qkv_norm_rope_fp4(x, None, **how)[0]
    hit = torch.zeros(n, H, dtype=torch.bool, device=DEV)
    for t, h, places in ((0, 0, range(d)), (0, 1, [0]), (1, 2, [d - 65]), (n - 1, H - 1, [17]),
                         (2, 0, [d - 1] + ([d - 1 - rope // 2 if half else d - 2] if rope else []))):
        hit[t, h] = True
        nan = torch.zeros(d, dtype=torch.bool, device=DEV)
        nan[list(places)] = True
        assert torch.equal(torch.isnan(got[t, h]), nan), (t, h, torch.isnan(got[t, h]).nonzero().tolist())
        assert (got[t, h][~nan] == 0).all()
    assert torch.equal(got[~hit], want[~hit])


@gpu
@pytest.mark.parametrize("half", [False, True])
def test_norm_rope_rows_near_the_ends_of_the_type(fk, half):
    """r below fp32's normal range (channels near 3e38), and rows of tiny channels: kv_out is exact."""
    n, d, rope = 4096, 512, 64
    x = torch.randn(n, d, generator=gen(72), device=DEV).clamp(-2, 2)
    x = (x * torch.where(torch.arange(n, device=DEV) % 2 == 0, 1.6e38, 1e-33)[:, None]).bfloat16()
    table, pos = table_of(64, rope), torch.arange(n, device=DEV) % 64
    _, kv = fk.qkv_norm_rope_fp4(None, x, positions=pos, cos_sin=table, rope_dim=rope, rope_half=half)
    want = bf16_of_f64(plain_norm_rope(x, None, pos, table, rope, half, 1e-6)[0])
    assert torch.equal(kv.float(), want.float())


@gpu
def test_norm_rope_strides_in_place_and_tokens_left_alone(fk):
    n, H, d, rope = 40, 6, 128, 64
    g = gen(5)
    fused = torch.randn(n, (H + 2) * d, generator=g, device=DEV).bfloat16()  # one projection's output
    q, kv = fused[:, : H * d].view(n, H, d), fused[:, H * d: (H + 1) * d]
    table, pos = table_of(100, rope), torch.randint(0, 100, (n,), generator=g, device=DEV)
    pos[3], pos[17] = -1, 100  # outside the table: these tokens are left alone
    gone = (pos < 0) | (pos >= 100)
    kw = dict(positions=pos, cos_sin=table, rope_dim=rope, rope_half=True)
    qo = torch.full((n, H, d), 9.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((n, d), 9.0, dtype=torch.bfloat16, device=DEV)
    fk.qkv_norm_rope_fp4(q, kv, q_out=qo, kv_out=ko, **kw)
    assert (qo[gone] == 9.0).all() and (ko[gone] == 9.0).all()
    keep = ~gone
    check_q(qo[keep], q[keep], None, pos[keep], table, rope, True, 1e-6)
    # heads outermost, and an output over its own input
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert qt.stride() != q.contiguous().stride()
    assert torch.equal(fk.qkv_norm_rope_fp4(qt, None, **kw)[0][keep], qo[keep])
    qi, ki = q.contiguous(), kv.contiguous()
    fk.qkv_norm_rope_fp4(qi, ki, q_out=qi, kv_out=ki, **kw)
    assert torch.equal(qi[keep], qo[keep]) and torch.equal(ki[keep], ko[keep])
    assert torch.equal(qi[gone], q[gone])
    # the KV row alone, queries alone, nothing at all
    assert torch.equal(fk.qkv_norm_rope_fp4(None, kv, **kw)[1][keep], ko[keep])
    none = fk.qkv_norm_rope_fp4(q[:0], kv[:0], positions=pos[:0], cos_sin=table, rope_dim=rope)
    assert none[0].shape == (0, H, d) and none[1].shape == (0, d)
    with pytest.raises(ValueError):
        fk.qkv_norm_rope_fp4(q, kv, rope_dim=32, positions=pos, cos_sin=table)
    with pytest.raises(ValueError):
        fk.qkv_norm_rope_fp4(q, kv[:5], **kw)
    with pytest.raises(ValueError):
        fk.qkv_norm_rope_fp4(q, None, packed=torch.empty(n, 64, dtype=torch.uint8, device=DEV), **kw)


# ----------------------------------------------------------------------------------------
# tree_attn_decode
# ----------------------------------------------------------------------------------------

def run_tree(fk, B, T, H, lens, drafts, cap, idx=None, seed=0, scale=512 ** -0.5, q=None, mask=None, cache=None, ws=None):
    packed, scales = make_cache(fk, B, cap, seed) if cache is None else cache
    if q is None:
        q = torch.randn(B, T, H, 512, generator=gen(seed + 1), device=DEV).bfloat16()
    if mask is None:
        mask = tree_masks(B, T, seed)
    out = torch.full((B, T, H, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, T, H), 5.0, device=DEV)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    nd = None if drafts is None else torch.tensor(drafts, dtype=torch.int32, device=DEV)
    ret = fk.tree_attn_decode(q, packed, scales, lt, mask, n_draft=nd, idx=idx, sm_scale=scale, out=out, lse=lse, ws=ws)
    assert ret[0] is out and ret[1] is lse
    dr = [T] * B if drafts is None else [max(0, min(x, T)) for x in drafts]
    check_tree(fk, q, packed, scales, lens, mask, dr, idx, scale, out, lse, f"B{B} T{T} H{H}")
    for b in range(B):  # tokens behind the last draft keep what was there
        assert (out[b, dr[b]:] == 3.0).all() and (lse[b, dr[b]:] == 5.0).all()
    return q, packed, scales, lt, mask, nd, out, lse


@gpu
@pytest.mark.parametrize("B, T, H, lens, drafts, cap", [
    (1, 1, 1, [0], None, 1),                       # the token alone
    (1, 1, 64, [1], None, 2),
    (1, 8, 64, [500], None, 508),
    (2, 3, 20, [63, 64], None, 80),                # a prefix that ends at, and one row before, a tile's end
    (3, 5, 12, [65, 127, 129], [5, 0, 2], 140),    # a sequence without drafts
    (2, 64, 8, [130, 0], [64, 63], 300),           # 64 drafts, one sequence without a prefix
    (1, 64, 128, [70], None, 134),                 # 8192 query rows
    (4, 7, 64, [1000, 3, 777, 64], [7, 7, 99, -5], 1007),  # draft counts outside [0, T]
    (1, 2, 6, [20000], None, 20002),               # few rows, a long prefix
    (1, 16, 64, [4093], None, 4100),               # the cache ends inside the drafts
    (2, 4, 16, [50, 9999], None, 60),              # a length behind the cache's end
    (33, 2, 3, [(i * 37) % 200 for i in range(33)], None, 202),
    (160, 1, 64, [(i * 29) % 150 for i in range(160)], None, 152),      # several short items to a cluster, 64 rows each
    (90, 3, 64, [(i * 53) % 700 for i in range(90)], [1 + i % 3 for i in range(90)], 800),  # 64, 128 and 192 rows
    (150, 2, 40, [(i * 61) % 900 for i in range(150)], None, 1000),     # parts of items, 80 rows each
])
def test_tree_dense(fk, B, T, H, lens, drafts, cap):
    run_tree(fk, B, T, H, lens, drafts, cap, seed=B + T + H)


@gpu
@pytest.mark.parametrize("B, T, H, lens, cap, K", [
    (1, 1, 64, [300], 310, 1), (3, 5, 64, [3000, 0, 40], 3005, 512), (2, 8, 20, [5000, 4999], 5008, 2048),
    (2, 33, 7, [100, 90], 140, 65), (1, 4, 16, [6000], 6004, 5000)])
def test_tree_selected(fk, B, T, H, lens, cap, K):
    idx = torch.full((B, K), -1, dtype=torch.int32, device=DEV)
    for b in range(B):
        k = min(K, lens[b])
        idx[b, :k] = torch.randperm(max(lens[b], 1), generator=gen(b), device=DEV)[:k].sort().values.int()
    run_tree(fk, B, T, H, lens, None, cap, idx=idx, seed=K)


@gpu
def test_tree_selection_in_any_order_with_holes_and_repeats(fk):
    B, T, H, cap, K = 2, 6, 24, 400, 200
    idx = torch.randint(0, 390, (B, K), generator=gen(1), device=DEV).int()
    idx[:, ::5] = -1
    idx[0, 1], idx[0, 2], idx[1, 3] = 2 ** 31 - 1, -2 ** 31, 391  # absent all the same
    idx[1, 64:128] = -1  # a whole tile absent
    idx[0, 10:20] = 7  # one row ten times
    run_tree(fk, B, T, H, [390, 390], [6, 4], cap, idx=idx, seed=9)


@gpu
def test_tree_masks_of_every_kind(fk):
    """Empty masks over an empty prefix (out 0, lse -inf), a token blind to itself, bits behind the
    last draft, the highest bit."""
    B, T, H = 2, 64, 5
    mask = tree_masks(B, T, 4)
    mask[:, 0] = 0
    mask[:, 1] = -1            # every bit
    mask[:, 2] = 1 << 1        # another draft only
    mask[:, 3] = -(1 << 63)    # the last draft only
    q, packed, scales, lt, mask, nd, out, lse = run_tree(fk, B, T, H, [0, 90], [64, 40], 160, mask=mask, seed=2)
    assert (out[0, 0] == 0).all() and torch.isneginf(lse[0, 0]).all()


@gpu
def test_tree_rows_nobody_sees_may_hold_anything(fk):
    """Drafted rows outside every mask, rows of the prefix outside the selection and rows behind the
    last draft hold bytes that stand for NaN."""
    B, T, H, cap = 2, 5, 64, 300
    packed, scales = make_cache(fk, B, cap, 6)
    lens, drafts = [200, 131], [5, 3]
    mask = torch.zeros(B, T, dtype=torch.int64, device=DEV)
    mask[:] = 0b00101  # drafts 1, 3, 4 are seen by nobody
    idx = torch.arange(0, 120, 2, dtype=torch.int32, device=DEV).repeat(B, 1)
    for b in range(B):
        keep = torch.zeros(cap, dtype=torch.bool, device=DEV)
        keep[idx[b].long()] = True
        keep[lens[b]], keep[lens[b] + 2] = True, True
        scales[b][~keep] = 0x7F
    run_tree(fk, B, T, H, lens, drafts, cap, idx=idx, mask=mask, cache=(packed, scales), seed=7)


@gpu
@pytest.mark.parametrize("scale", [1.0, 0.3, -0.05, 0.0])
def test_tree_large_logits_that_grow_along_the_prefix(fk, scale):
    """Logits up to a few thousand whose running maximum keeps moving, in every tile and head at
    another place."""
    B, T, H, n = 1, 3, 50, 1500
    g = gen(11)
    x = torch.randn(n + T, 512, generator=g, device=DEV)
    x *= torch.linspace(0.01, 4.0, n + T, device=DEV)[:, None]
    packed = torch.empty(1, n + T, 256, dtype=torch.uint8, device=DEV)
    scales = torch.empty(1, n + T, 32, dtype=torch.uint8, device=DEV)
    fk.kv_quant_fp4(x.bfloat16(), packed[0], scales[0])
    q = torch.randn(B, T, H, 512, generator=g, device=DEV) * torch.logspace(-3, 1, H, device=DEV)[:, None]
    run_tree(fk, B, T, H, [n], None, n + T, cache=(packed, scales), q=q.bfloat16(), scale=scale, seed=1)


@gpu
def test_tree_extreme_queries(fk):
    """Zero queries (a plain mean), one loud channel, queries near bf16's ends."""
    B, T, H, n = 1, 2, 8, 700
    q = torch.randn(B, T, H, 512, generator=gen(3), device=DEV)
    q[0, 0, 0] = 0.0
    q[0, 0, 1, 1:] = 0.0
    q[0, 0, 2] *= 1e-30
    q[0, 0, 3, 7] = 300.0
    run_tree(fk, B, T, H, [n], None, n + T, q=q.bfloat16(), scale=0.02, seed=3)
    run_tree(fk, B, T, H, [n], None, n + T, q=(q * 1e30).bfloat16(), scale=2e-32, seed=3)


@gpu
@pytest.mark.parametrize("n", [40, 900])  # (whole items, and items in parts)
def test_tree_a_nan_row_reaches_only_those_who_see_it(fk, n):
    """A drafted row whose scale is NaN, as the quantizer writes for a row with NaN: NaN for the tokens
    that see it, nothing for the others."""
    B, T, H = 1, 4, 40
    packed, scales = make_cache(fk, B, n + T, 16)
    mask = torch.tensor([[0b0001, 0b0011, 0b0101, 0b1101]], dtype=torch.int64, device=DEV)
    q = torch.randn(B, T, H, 512, generator=gen(17), device=DEV).bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    want, wl = fk.tree_attn_decode(q, packed, scales, lens, mask, sm_scale=0.04)
    bad = scales.clone()
    bad[0, n + 2, 5] = 0x7F
    bad[0, n + 2, 9] = 0xFF
    out, lse = fk.tree_attn_decode(q, packed, bad, lens, mask, sm_scale=0.04)
    assert torch.equal(out[:, :2], want[:, :2]) and torch.equal(lse[:, :2], wl[:, :2])
    assert torch.isnan(out[:, 2:]).all() and torch.isnan(lse[:, 2:]).all()


@gpu
@pytest.mark.parametrize("n", [40, 900])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_tree_queries_that_are_not_finite(fk, n, value):
    """NaN for their own head (softmax of infinite logits has no value), the others as they were; a token
    that sees nothing gives 0 all the same."""
    B, T, H = 2, 2, 70
    packed, scales = make_cache(fk, B, n + T, 18)
    mask = torch.tensor([[1, 2], [0, 3]], dtype=torch.int64, device=DEV)
    q = torch.randn(B, T, H, 512, generator=gen(19), device=DEV).bfloat16()
    lens = torch.tensor([n, 0], dtype=torch.int32, device=DEV)
    want, wl = fk.tree_attn_decode(q, packed, scales, lens, mask, sm_scale=0.04)
    x = q.clone()
    hit = torch.zeros(B, T, H, dtype=torch.bool, device=DEV)
    for b, t, h, c in [(0, 0, 0, 0), (0, 1, 69, 511), (0, 1, 3, 100), (1, 0, 5, 7), (1, 1, 64, 256)]:
        x[b, t, h, c] = value
        hit[b, t, h] = (b, t) != (1, 0)
    out, lse = fk.tree_attn_decode(x, packed, scales, lens, mask, sm_scale=0.04)
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wl[~hit])
    assert (out[1, 0] == 0).all() and torch.isneginf(lse[1, 0]).all()


@gpu
def test_tree_binding_checks(fk):
    q, packed, scales, lt, mask, nd, out, lse = run_tree(fk, 1, 2, 4, [10], None, 12)
    o, l = fk.tree_attn_decode(q, packed, scales, lt, mask, sm_scale=512 ** -0.5)
    assert torch.equal(o, out) and torch.equal(l, lse)
    assert fk.tree_attn_decode(q, packed, scales, lt, mask, want_lse=False)[1] is None
    with pytest.raises(ValueError):
        fk.tree_attn_decode(q[0], packed, scales, lt, mask)
    with pytest.raises(ValueError):
        fk.tree_attn_decode(q, packed[:, :, :128], scales, lt, mask)
    with pytest.raises(ValueError):
        fk.tree_attn_decode(q, packed, scales, lt, mask[:, :1])
    with pytest.raises(TypeError):
        fk.tree_attn_decode(q, packed, scales, lt.long(), mask)
    with pytest.raises(ValueError):
        fk.tree_attn_decode(q, packed, scales, lt, mask, out=out[:, :1])
    with pytest.raises(fk.Fp4kvError):
        fk.tree_attn_decode(q, packed, scales, lt, mask, ws=torch.zeros(128, dtype=torch.uint8, device=DEV))


@gpu
def test_tree_same_bits_every_time_and_from_a_replayed_graph(fk):
    """Nothing depends on timing; graphs that share a workspace replay one after another; lengths
    are read at replay."""
    B, T, H, cap = 3, 6, 64, 5000
    ws = fk.alloc_workspace(fk.workspace_bytes(fk.OP_TREE_ATTN, B, cap, T * H, 0), DEV)
    q, packed, scales, lt, mask, nd, out, lse = run_tree(fk, B, T, H, [4990, 17, 2222], [6, 6, 4], cap, seed=5, ws=ws)
    ref = out.clone(), lse.clone()
    for _ in range(3):
        fk.tree_attn_decode(q, packed, scales, lt, mask, n_draft=nd, sm_scale=512 ** -0.5, ws=ws, out=out, lse=lse)
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    graphs, outs = [], []
    torch.cuda.synchronize()
    for i in range(2):
        o, l = torch.full_like(out, 3.0), torch.full_like(lse, 5.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fk.tree_attn_decode(q, packed, scales, lt, mask, n_draft=nd, sm_scale=512 ** -0.5, ws=ws, out=o, lse=l)
        graphs.append(g)
        outs.append((o, l))
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, ref[0]) and torch.equal(l, ref[1])
    lt.copy_(torch.tensor([100, 3000, 0], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    check_tree(fk, q, packed, scales, lt.tolist(), mask, [6, 6, 4], None, 512 ** -0.5, *outs[0])
    assert fk.workspace_status(ws) == 0


# ----------------------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------------------

@gpu
def test_a_step_of_verifying_drafts(fk):
    """Norm, rotation and write of the drafts' rows behind the prefix, attention of the tree, the
    accepted row read back; the same tokens decoded one by one with sparse_attn_decode agree."""
    B, T, H, d, rope, n = 3, 4, 64, 512, 64, 600
    cap = n + T
    packed, scales = make_cache(fk, B, cap, 21)
    lens = [n, 333, 64]
    g = gen(22)
    qkv = torch.randn(B * T, (H + 1) * d, generator=g, device=DEV).bfloat16()
    w = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).bfloat16()
    table = table_of(cap, rope)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    pos = (lt.long()[:, None] + torch.arange(T, device=DEV)).view(-1)
    dst = pos + torch.arange(B, device=DEV).repeat_interleave(T) * cap
    q, _ = fk.qkv_norm_rope_fp4(qkv[:, : H * d].view(B * T, H, d), qkv[:, H * d:], positions=pos, cos_sin=table,
                                rope_dim=rope, q_weight=w, kv_weight=w, packed=packed, scales=scales, dst_row=dst)
    chain = torch.tensor([[(1 << (t + 1)) - 1 for t in range(T)]] * B, dtype=torch.int64, device=DEV)
    scale = d ** -0.5
    out, lse = fk.tree_attn_decode(q.view(B, T, H, d), packed, scales, lt, chain, sm_scale=scale)
    rows = fk.kv_dequant_fp4(packed, scales, src_row=dst)
    check_tree(fk, q.view(B, T, H, d), packed, scales, lens, chain, [T] * B, None, scale, out, lse)
    y = plain_norm_rope(qkv[:, H * d:], w, pos, table, rope, False, 1e-6)[0]
    op, os_ = O.kv_quant_fp4(P.to_f64(bf16_of_f64(y)))
    assert np.array_equal(rows.double().cpu().numpy(), O.kv_dequant_fp4(op, os_))
    idx = torch.arange(cap, dtype=torch.int32, device=DEV).repeat(B, 1)
    for t in range(T):
        one, l1 = fk.sparse_attn_decode(q.view(B, T, H, d)[:, t].contiguous(), packed, scales, lt + t + 1, idx, scale)
        assert (l1 - lse[:, t]).abs().max() <= 1e-4
        assert (one - out[:, t].float()).abs().max() <= 5e-3 + 2.0 ** -8 * one.abs().max()


@gpu
def test_norm_output_feeds_the_attention_at_once(fk):
    """No synchronisation between the kernel that makes q (and the cache row) and those that read
    them, many times over, also on a side stream."""
    n, H, d = 600, 64, 512
    packed, scales = make_cache(fk, 1, n, 31)
    idx = torch.arange(256, dtype=torch.int32, device=DEV).view(1, -1)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    ws = fk.alloc_workspace(fk.workspace_bytes(fk.OP_SPARSE_ATTN, 1, n, H, 256), DEV)
    raw = [torch.randn(1, H, d, generator=gen(40 + i), device=DEV).bfloat16() for i in range(8)]
    q = torch.empty(1, H, d, dtype=torch.bfloat16, device=DEV)
    outs = [torch.empty(1, H, d, device=DEV) for _ in raw]
    want = []
    for x in raw:
        y, _ = fk.qkv_norm_rope_fp4(x, None)
        torch.cuda.synchronize()
        want.append(fk.sparse_attn_decode(y, packed, scales, lens, idx, 0.04, ws=ws, want_lse=False)[0].clone())
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(5):
                for x, o in zip(raw, outs):
                    fk.qkv_norm_rope_fp4(x, None, q_out=q)
                    fk.sparse_attn_decode(q, packed, scales, lens, idx, 0.04, ws=ws, out=o, want_lse=False)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@gpu
@pytest.mark.parametrize("n", [200, 900])  # (items that stay whole, and items that are joined by a second launch)
def test_tree_output_feeds_the_attention_at_once(fk, n):
    """The tree's output as the query of sparse_attn_decode, with nothing between the two launches."""
    H, d = 64, 512
    packed, scales = make_cache(fk, 1, n, 33)
    idx = torch.arange(128, dtype=torch.int32, device=DEV).view(1, -1)
    lens = torch.tensor([n - 1], dtype=torch.int32, device=DEV)
    mask = torch.ones(1, 1, dtype=torch.int64, device=DEV)
    ws = fk.alloc_workspace(fk.workspace_bytes(fk.OP_SPARSE_ATTN, 1, n, H, 128), DEV)
    tws = fk.alloc_workspace(fk.workspace_bytes(fk.OP_TREE_ATTN, 1, n, H, 0), DEV)
    raw = [torch.randn(1, 1, H, d, generator=gen(60 + i), device=DEV).bfloat16() for i in range(8)]
    mid = torch.empty(1, 1, H, d, dtype=torch.bfloat16, device=DEV)
    outs = [torch.empty(1, H, d, device=DEV) for _ in raw]

    def step(x, o, wait):
        fk.tree_attn_decode(x, packed, scales, lens, mask, sm_scale=0.04, out=mid, ws=tws)
        if wait:
            torch.cuda.synchronize()
        fk.sparse_attn_decode(mid.view(1, H, d), packed, scales, lens, idx, 0.04, ws=ws, out=o, want_lse=False)

    want = []
    for x, o in zip(raw, outs):
        step(x, o, True)
        torch.cuda.synchronize()
        want.append(o.clone())
    for _ in range(5):
        for x, o in zip(raw, outs):
            step(x, o, False)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def at_offset(t, nbytes):
    """t's contents in a buffer that starts nbytes behind an allocation's start."""
    raw = torch.empty(t.numel() * t.element_size() + nbytes, dtype=torch.uint8, device=t.device)
    out = raw[nbytes:].view(t.dtype).view(t.shape)
    out.copy_(t)
    return out


@gpu
@pytest.mark.parametrize("B, T, H, cap", [(8, 9, 64, 700), (74, 2, 64, 800), (75, 2, 64, 800), (72, 1, 5, 1100), (37, 4, 64, 1216), (37, 4, 64, 1217)])
def test_tree_batches_on_either_side_of_the_sharing_rule(fk, B, T, H, cap):
    """Items whole or shared by how evenly they fill the GPU, with lengths that differ widely."""
    lens = [(cap - T) * ((5 * b) % 9) // 8 for b in range(B)]
    run_tree(fk, B, T, H, lens, [T - b % (T + 1) for b in range(B)], cap, seed=13)


@gpu
@pytest.mark.parametrize("n, H, d, rope, half", [(2367, 0, 512, 64, True), (2368, 0, 512, 64, False), (2368, 0, 1024, 64, False), (4800, 0, 128, 64, True),
                                                 (37, 128, 64, 32, False), (150, 63, 512, 64, True), (300, 64, 96, 0, False), (297, 33, 256, 256, False)])
def test_norm_rope_on_either_side_of_its_splits(fk, n, H, d, rope, half):
    g = gen(n + d)
    kv = torch.randn(n, d, generator=g, device=DEV).bfloat16()
    q = torch.randn(n, H, d, generator=g, device=DEV).bfloat16() if H else None
    table, pos = table_of(100, rope) if rope else None, torch.arange(n, device=DEV) % 100
    qo, ko = fk.qkv_norm_rope_fp4(q, kv, positions=pos if rope else None, cos_sin=table, rope_dim=rope, rope_half=half)
    if H:
        check_q(qo, q, None, pos, table, rope, half, 1e-6)
    assert torch.equal(ko, bf16_of_f64(plain_norm_rope(kv, None, pos, table, rope, half, 1e-6)[0]))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [9471, 9473, 18944, 18945])
def test_dequant_on_either_side_of_its_split(fk, n, dtype):
    packed, scales = make_cache(fk, 1, 900, 14)
    rows = torch.randint(-1, 901, (n,), generator=gen(n), device=DEV)
    v = cache_values(packed[0], scales[0]).to(DEV)
    want = torch.where(((rows >= 0) & (rows < 900))[:, None], v[rows.clamp(0, 899)], 0.0)
    assert torch.equal(fk.kv_dequant_fp4(packed, scales, src_row=rows, dtype=dtype).double(), want)


@gpu
def test_bases_at_the_least_alignment(fk):
    """The same bits from tensors that have only the alignment that the calls ask for."""
    B, T, H, n, d = 2, 3, 50, 700, 512
    packed, scales = make_cache(fk, B, n + T, 51)
    p2, s2 = at_offset(packed, 16), at_offset(scales, 16)
    lens = torch.tensor([n, 130], dtype=torch.int32, device=DEV)
    mask = tree_masks(B, T, 3)
    q = torch.randn(B, T, H, d, generator=gen(52), device=DEV).bfloat16()
    for idx in (None, torch.randint(0, n, (B, 201), generator=gen(53), device=DEV).int()):
        out, lse = fk.tree_attn_decode(q, packed, scales, lens, mask, idx=idx, sm_scale=0.04)
        o2, l2 = fk.tree_attn_decode(at_offset(q, 16), p2, s2, lens, mask, idx=None if idx is None else at_offset(idx, 4),
                                     sm_scale=0.04, out=at_offset(torch.zeros_like(q), 16), lse=at_offset(lse * 0, 4))
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    rows = torch.randint(-3, B * (n + T) + 3, (333,), generator=gen(54), device=DEV)
    for dtype, pad in ((torch.bfloat16, 8), (torch.float32, 4)):
        want = fk.kv_dequant_fp4(packed, scales, src_row=rows, dtype=dtype)
        wide = at_offset(torch.zeros(333, d + pad, dtype=dtype, device=DEV), 16)
        got = fk.kv_dequant_fp4(p2, at_offset(scales, 1), src_row=at_offset(rows, 8), out=wide[:, :d])
        assert torch.equal(got, want) and (wide[:, d:] == 0).all()
    x = torch.randn(300, d, generator=gen(55), device=DEV).bfloat16()
    c1, c2 = torch.zeros(300, d // 2, dtype=torch.uint8, device=DEV), torch.zeros(300, d // 16, dtype=torch.uint8, device=DEV)
    c3, c4 = at_offset(c1, 8), at_offset(c2, 1)
    fk.qkv_norm_rope_fp4(None, x, packed=c1, scales=c2)
    fk.qkv_norm_rope_fp4(None, at_offset(x, 16), packed=c3, scales=c4)
    assert torch.equal(c3, c1) and torch.equal(c4, c2)


@gpu
def test_a_cache_of_more_than_2_gib(fk):
    """Rows behind 2^31 bytes: written, read back and attended."""
    cap, d, H, T = 8_500_000, 512, 64, 2
    packed = torch.zeros(1, cap, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(1, cap, d // 16, dtype=torch.uint8, device=DEV)
    small_p, small_s = make_cache(fk, 1, 300 + T, 56)
    at = torch.cat([torch.arange(150, device=DEV), torch.arange(cap - T - 150, cap, device=DEV)])
    packed[0, at], scales[0, at] = small_p[0], small_s[0]
    x = torch.randn(T, d, generator=gen(57), device=DEV).bfloat16()
    fk.qkv_norm_rope_fp4(None, x, packed=packed, scales=scales, dst_row=at[-T:].contiguous())
    fk.qkv_norm_rope_fp4(None, x, packed=small_p, scales=small_s, dst_row=torch.arange(300, 300 + T, device=DEV))
    assert torch.equal(fk.kv_dequant_fp4(packed, scales, src_row=at), fk.kv_dequant_fp4(small_p, small_s))
    q = torch.randn(1, T, H, d, generator=gen(58), device=DEV).bfloat16()
    mask = torch.tensor([[1, 3]], dtype=torch.int64, device=DEV)
    far = fk.tree_attn_decode(q, packed, scales, torch.tensor([cap - T], dtype=torch.int32, device=DEV), mask,
                              idx=at[:300].int().view(1, -1), sm_scale=0.04)
    near = fk.tree_attn_decode(q, small_p, small_s, torch.tensor([300], dtype=torch.int32, device=DEV), mask,
                               idx=torch.arange(300, dtype=torch.int32, device=DEV).view(1, -1), sm_scale=0.04)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])


@gpu
def test_two_streams_at_once_and_nothing_drafted(fk):
    """Calls with their own workspaces overlap on two streams; a batch without a single draft writes nothing."""
    B, T, H, n = 2, 4, 64, 3000
    packed, scales = make_cache(fk, B, n + T, 59)
    lens = torch.tensor([n, 1700], dtype=torch.int32, device=DEV)
    mask = tree_masks(B, T, 5)
    q = [torch.randn(B, T, H, 512, generator=gen(60 + i), device=DEV).bfloat16() for i in range(2)]
    want = [fk.tree_attn_decode(x, packed, scales, lens, mask, sm_scale=0.04) for x in q]
    ws = [fk.alloc_workspace(fk.workspace_bytes(fk.OP_TREE_ATTN, B, n + T, T * H, 0), DEV) for _ in q]
    got = [(torch.zeros_like(o), torch.zeros_like(l)) for o, l in want]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                fk.tree_attn_decode(q[i], packed, scales, lens, mask, sm_scale=0.04, ws=ws[i], out=got[i][0], lse=got[i][1])
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
    o, l = got[0][0].fill_(3.0), got[0][1].fill_(4.0)
    none = torch.tensor([0, -5], dtype=torch.int32, device=DEV)
    fk.tree_attn_decode(q[0], packed, scales, lens, mask, n_draft=none, ws=ws[0], out=o, lse=l)
    assert (o == 3.0).all() and (l == 4.0).all() and all(fk.workspace_status(w) == 0 for w in ws)


@gpu
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n, H, d", [(520, 64, 512), (2400, 0, 512), (2400, 0, 128), (2400, 0, 1024), (3, 64, 512)])
def test_norm_rope_in_place_at_every_split(fk, n, H, d, half):
    """Rows written over themselves give the bits of separate outputs."""
    q = torch.randn(n, H, d, generator=gen(81), device=DEV).bfloat16() if H else None
    kv = torch.randn(n, d, generator=gen(82), device=DEV).bfloat16()
    table, pos = table_of(50, 64), torch.arange(n, device=DEV) % 50
    how = dict(positions=pos, cos_sin=table, rope_dim=64, rope_half=half)
    qw, kw = fk.qkv_norm_rope_fp4(q, kv, **how)
    qo, ko = fk.qkv_norm_rope_fp4(q, kv, q_out=q, kv_out=kv, **how)
    assert torch.equal(ko, kw) and ko.data_ptr() == kv.data_ptr()
    assert H == 0 or (torch.equal(qo, qw) and qo.data_ptr() == q.data_ptr())


@gpu
@pytest.mark.parametrize("B, T, n", [(2, 4, 300), (16, 16, 1500)])  # (plain launches and whole items; dependent ones and a merge)
def test_a_captured_step_replays_with_what_the_tensors_hold_then(fk, B, T, n):
    """Norm and write, tree, read-back in one graph: replayed after every input has changed, equal to the calls
    made one by one."""
    H, d, rope, cap = 64, 512, 64, n + T
    table = table_of(cap, rope)
    ws = fk.alloc_workspace(fk.workspace_bytes(fk.OP_TREE_ATTN, B, cap, T * H, 0), DEV)
    packed, scales = make_cache(fk, B, cap, 83)
    x = torch.empty(B * T, (H + 1) * d, dtype=torch.bfloat16, device=DEV)
    lens, mask = torch.empty(B, dtype=torch.int32, device=DEV), torch.empty(B, T, dtype=torch.int64, device=DEV)
    pos, dst = torch.empty(B * T, dtype=torch.int64, device=DEV), torch.empty(B * T, dtype=torch.int64, device=DEV)
    q = torch.empty(B, T, H, d, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(B, T, H, device=DEV)
    rows = torch.empty(B * T, d, dtype=torch.bfloat16, device=DEV)

    def fill(seed):
        x.copy_(torch.randn(x.shape, generator=gen(seed), device=DEV))
        lens.copy_(torch.randint(0, n + 1, (B,), generator=gen(seed + 1), device=DEV))
        mask.copy_(tree_masks(B, T, seed))
        pos.copy_((lens.long()[:, None] + torch.arange(T, device=DEV)).view(-1))
        dst.copy_(pos + torch.arange(B, device=DEV).repeat_interleave(T) * cap)

    def step():
        fk.qkv_norm_rope_fp4(x[:, : H * d].view(B * T, H, d), x[:, H * d:], positions=pos, cos_sin=table, rope_dim=rope,
                             packed=packed, scales=scales, dst_row=dst, q_out=q.view(B * T, H, d))
        fk.tree_attn_decode(q, packed, scales, lens, mask, sm_scale=0.04, ws=ws, out=out, lse=lse)
        fk.kv_dequant_fp4(packed, scales, src_row=dst, out=rows)

    fill(90)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (91, 95):
        fill(seed)
        keep = packed.clone(), scales.clone()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q, out, lse, rows, packed, scales)]
        packed.copy_(keep[0]), scales.copy_(keep[1])
        for t in (q, out, lse, rows):
            t.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (q, out, lse, rows, packed, scales)):
            assert torch.equal(a, b)
    assert fk.workspace_status(ws) == 0


# ----------------------------------------------------------------------------------------
# what the probabilities keep
# ----------------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("B, T, H, n", [(1, 2, 64, 2), (3, 2, 5, 6), (1, 2, 64, 700), (2, 4, 64, 3000)])
def test_tree_rows_that_cancel(fk, B, T, H, n):
    """Rows in pairs w, -w of nearly the same probability: out is the small difference of large terms, so what a
    probability loses shows beside the output's bf16. Queries have one channel, whose logits (|z| < 0.02) are
    exact but for fp32's rounding. A probability: its exponent in fp32, at most 16 in size, 2^-21; ex2 2^-22; its two
    parts 2^-21; the row's sum the same again: together below 2^-18 of A = sum p |v|. The accumulator takes two steps for
    every 16 rows, and as many joins as there are parts (at most one per two tiles), 2^-23 each. A probability in
    fp16 alone would be off by up to 2^-12."""
    cap = n + T
    g = gen(100 + n)
    packed = torch.randint(0, 256, (B, cap // 2, 1, 256), generator=g, device=DEV).to(torch.uint8).repeat(1, 1, 2, 1)
    packed[:, :, 1] ^= 0x88                     # the other sign
    packed = packed.reshape(B, cap, 256)
    packed[:, :, :8] = torch.randint(0, 256, (B, cap, 8), generator=g, device=DEV).to(torch.uint8)  # channels 0 .. 15 apart
    scales = torch.randint(0x30, 0x58, (B, cap // 2, 1, 32), generator=g, device=DEV).to(torch.uint8).repeat(1, 1, 2, 1).reshape(B, cap, 32)
    scales[:, :, 0] = 0x38                      # channels 0 .. 15: values up to 6
    q = torch.zeros(B, T, H, 512, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = (1 + torch.arange(H, device=DEV) / 64).bfloat16()
    mask = torch.full((B, T), (1 << T) - 1, dtype=torch.int64, device=DEV)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    scale = 2.0 ** -10
    out, lse = fk.tree_attn_decode(q, packed.contiguous(), scales.contiguous(), lens, mask, sm_scale=scale)
    for b in range(B):
        v = cache_values(packed[b], scales[b])
        p = torch.softmax(q[b].double().cpu() @ v.T * scale, -1)
        want, A = p @ v, p @ v.abs()
        steps = 2 * ((cap + 15) // 16) + (cap + 127) // 128
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -18 + steps * 2.0 ** -23) * A
        off = (out[b].double().cpu() - want).abs()
        assert (off <= tol).all(), f"off by {(off / A).max():.2e} of the terms, {((off - tol) / A).max():.2e} too much"


@gpu
@pytest.mark.parametrize("heavy", [0.0, 0.02])
def test_tree_keeps_the_attention_tolerance(fk, heavy):
    """The library's bounds on its attention, before the rounding to bf16: 5e-3 in every value, lse within 1e-4, also
    where one row in fifty is a hundred times louder (with queries a hundred times softer, so that several of those
    rows share the sum); and sparse_attn_decode's own values, rounded."""
    B, T, H, n, d = 2, 3, 64, 1500, 512
    cap = n + T
    x = P.kv_rows_dev(77, 0, B, cap, d, torch.device(DEV), heavy=heavy)
    packed, scales = torch.empty(B, cap, d // 2, dtype=torch.uint8, device=DEV), torch.empty(B, cap, d // 16, dtype=torch.uint8, device=DEV)
    fk.kv_quant_fp4(x.view(-1, d), packed.view(-1, d // 2), scales.view(-1, d // 16))
    q = torch.stack([synth.attn_query(77, t, B, H, d, device=torch.device(DEV)) for t in range(T)], 1)
    q = (q * (0.01 if heavy else 1.0)).contiguous()
    mask = torch.full((B, T), 7, dtype=torch.int64, device=DEV)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    out, lse = fk.tree_attn_decode(q, packed, scales, lens, mask, sm_scale=1.0)
    for b in range(B):
        v = cache_values(packed[b], scales[b])
        z = q[b].double().cpu() @ v.T
        want = torch.softmax(z, -1) @ v
        off = (out[b].double().cpu() - want).abs()
        assert (off <= P.ATTN_MAX_ABS + 2.0 ** -8 * (want.abs() + P.ATTN_MAX_ABS)).all(), f"off by {off.max():.2e}"
        assert (lse[b].double().cpu() - torch.logsumexp(z, -1)).abs().max() <= P.LSE_ABS
    idx = torch.arange(cap, dtype=torch.int32, device=DEV).repeat(B, 1)
    one, l1 = fk.sparse_attn_decode(q[:, 0].contiguous(), packed, scales, lens + T, idx, 1.0)
    assert ((one - out[:, 0].float()).abs() <= 2 * P.ATTN_MAX_ABS + 2.0 ** -8 * one.abs() + 2.0 ** -8 * P.ATTN_MAX_ABS).all()
    assert (l1 - lse[:, 0]).abs().max() <= 2 * P.LSE_ABS


@gpu
@pytest.mark.parametrize("n", [100, 3000])  # (whole items, and items in parts)
@pytest.mark.parametrize("loud, scale", [(1.0, 1e3), (1e3, 1e4), (1e6, 1e6), (1e20, 1e-3), (1e37, 1e3), (1e-30, 3e38), (1e3, -1e7)])
def test_tree_logits_beyond_what_fp32_counts(fk, n, loud, scale):
    """Logits from 1e5 to past fp32's range: every head gives the one row that wins, which is exact in bf16 (6 bits);
    lse is the winner's logit. Heads whose second row is within what a logit may be off by, and 40, are left out: the
    other rows' weights are together below 3003 e^-40 < 2^-46, their values below 2^12, so out is off by at most 2^-33
    (less than bf16's step at any value of the cache but 0)."""
    B, T, H = 1, 3, 64
    packed, scales = make_cache(fk, B, n + T, 120)
    q = (torch.randn(B, T, H, 512, generator=gen(121), device=DEV) * loud).bfloat16()
    mask = torch.full((B, T), 7, dtype=torch.int64, device=DEV)
    out, lse = fk.tree_attn_decode(q, packed, scales, torch.tensor([n], dtype=torch.int32, device=DEV), mask, sm_scale=scale)
    v = cache_values(packed[0], scales[0])
    qq = q[0].double().cpu()
    scale32 = float(np.float32(scale))
    z = qq @ v.T * scale32
    dz = 2.0 ** -16 * abs(scale32) * (qq.abs() @ v.abs().T).amax(-1)
    top = z.topk(2, -1)
    sure = top.values[..., 0] - top.values[..., 1] > 2 * dz + 40.0
    assert sure.double().mean() > 0.9
    assert torch.isfinite(out).all()
    assert ((out[0].double().cpu() - v[top.indices[..., 0]]).abs()[sure] <= 2.0 ** -33).all()
    l, want = lse[0].double().cpu()[sure], top.values[..., 0][sure]
    far = want.abs() > 3.4e38  # (past the type)
    assert torch.equal(l[far], torch.sign(want[far]) * np.inf)
    assert ((l - want).abs() <= dz[sure] + 2.0 ** -21 * want.abs())[~far].all()


@gpu
@pytest.mark.parametrize("spread", [True, False])
@pytest.mark.parametrize("B, T, H, n", [(1, 64, 128, 1_000_000), (80, 1, 5, 120_000), (1, 64, 128, 16_800), (3, 64, 64, 16_400)])
def test_tree_long_prefixes_do_not_drift(fk, B, T, H, n, spread):
    """Every row has 1.0 in its last 496 channels, so out is 1.0 there, whatever the probabilities are (n of them, of many
    sizes or all but one of the same): what a long sum of them loses is lost by the values or by the row's sum alone,
    and shows as soon as it passes 2^-9. O is summed over at most 256 tiles (2,048 steps, each off by up to 2^-23: 2^-12)
    and then with rounding, the sum of a row over 2,048 terms a thread (half of 2^-23 each) and then likewise."""
    cap = n + T
    g = gen(130)
    packed = torch.full((B, cap, 256), 0x22, dtype=torch.uint8, device=DEV)
    packed[:, :, :8] = torch.randint(0, 256, (B, cap, 8), generator=g, device=DEV).to(torch.uint8) if spread else 0x11
    if not spread:
        packed[:, 5, :8] = 0x77  # one row's logit is larger
    scales = torch.full((B, cap, 32), 0x38, dtype=torch.uint8, device=DEV)
    q = torch.zeros(B, T, H, 512, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = (1 + torch.arange(H, device=DEV) / 128).bfloat16()
    mask = torch.ones(B, T, dtype=torch.int64, device=DEV)
    out, lse = fk.tree_attn_decode(q, packed, scales, torch.full((B,), n, dtype=torch.int32, device=DEV), mask, sm_scale=0.37)
    assert (out[..., 16:] == 1.0).all(), f"{out[..., 16:].min().item()} .. {out[..., 16:].max().item()}"
    for b in range(0, B, 40):
        v0 = cache_values(packed[b, :, :8].repeat(1, 32), scales[b])[: n + 1, 0]
        for h in (0, H - 1):
            z = v0 * q[b, 0, h, 0].double().cpu() * float(np.float32(0.37))
            p = torch.softmax(z, -1)
            assert abs(lse[b, 0, h].item() - torch.logsumexp(z, -1).item()) <= 2.0 ** -11
            assert abs(out[b, 0, h, 0].item() - (p @ v0).item()) <= 2.0 ** -8 * abs((p @ v0).item()) + 2.0 ** -10 * (p @ v0.abs()).item()


@gpu
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("B, T, H, n", [(1, 64, 128, 40_000), (2, 33, 128, 33_000), (1, 37, 128, 80_000)])  # (whole items, and parts)
def test_tree_references_that_move_between_flushes(fk, B, T, H, n, rising):
    """Logits that grow (or shrink) by 2^13 in all along a prefix of several times 256 tiles: what has been put
    aside is scaled down again and again, or stays. The bound of test_tree_rows_that_cancel, with 2,048 steps."""
    cap = n + T
    g = gen(140)
    packed = torch.randint(0, 256, (B, cap, 256), generator=g, device=DEV).to(torch.uint8)
    scales = torch.randint(0x30, 0x40, (B, cap, 32), generator=g, device=DEV).to(torch.uint8)
    ramp = torch.linspace(0x08, 0x60, cap, device=DEV)
    scales[:, :, 0] = (ramp if rising else ramp.flip(0)).to(torch.uint8)
    packed[:, :, 0] = 0x77
    q = torch.zeros(B, T, H, 512, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = (1 + torch.arange(H, device=DEV) / 128).bfloat16()
    mask = tree_masks(B, T, 8)
    out, lse = fk.tree_attn_decode(q, packed, scales, torch.full((B,), n, dtype=torch.int32, device=DEV), mask, sm_scale=0.11)
    for b in range(B):
        v = cache_values(packed[b], scales[b]).to(DEV)
        for t in (0, T - 1):
            z = v[:, 0] * float(np.float32(0.11)) * q[b, t, :, :1].double()
            m = int(mask[b, t])
            z[:, n:][:, [not m >> j & 1 for j in range(T)]] = -np.inf
            p = torch.softmax(z, -1)
            want, A = p @ v, p @ v.abs()
            off = (out[b, t].double() - want).abs()
            assert (off <= 2.0 ** -8 * want.abs() + (2.0 ** -17 + 2.0 ** -12) * A).all(), f"{(off / A).max():.2e}"
            assert ((lse[b, t].double() - torch.logsumexp(z, -1)).abs() <= 2.0 ** -11 + 2.0 ** -21 * torch.logsumexp(z, -1).abs()).all()


@gpu
def test_one_workspace_for_several_ops(fk):
    """Attention and tree calls may follow any op on a workspace; an indexer call follows another op, or other sizes,
    after workspace_init."""
    B, T, H, cap, K, dev = 2, 4, 64, 6000, 512, torch.device(DEV)
    lens = torch.tensor([cap - T, 4321], dtype=torch.int32, device=dev)
    packed, scales = make_cache(fk, B, cap, 160)
    mask = tree_masks(B, T, 9)
    q = torch.randn(B, T, H, 512, generator=gen(161), device=dev).bfloat16()
    qi, w = synth.indexer_query(5, 0, B, 32, device=dev)
    keys = P.keys_dev(5, B, cap, True, dev)
    need = [fk.workspace_bytes(fk.OP_TREE_ATTN, B, cap, T * H, top_k) for top_k in (0, K)]
    need += [fk.workspace_bytes(fk.OP_INDEXER_TOPK, B, cap, 32, K), fk.workspace_bytes(fk.OP_SPARSE_ATTN, B, cap, H, K)]
    ws = fk.alloc_workspace(max(need), dev)

    def select(ws=None, n=cap):
        return fk.indexer_topk(qi, w, keys[:, :n].contiguous(), lens.clamp(max=n), K, ws=ws)

    def tree(idx, ws=None):
        return fk.tree_attn_decode(q, packed, scales, lens, mask, idx=idx, sm_scale=0.04, ws=ws)

    def sparse(idx, ws=None):
        return fk.sparse_attn_decode(q[:, 0].contiguous(), packed, scales, lens, idx, 0.04, ws=ws)

    idx, small = select(), select(n=3000)
    dense, chosen, one = tree(None), tree(idx), sparse(idx)
    for _ in range(2):
        for n, want in ((cap, idx), (3000, small)):
            fk.workspace_init(ws)
            for _ in range(2):
                assert torch.equal(select(ws, n), want)
            for got, ref in ((tree(None, ws), dense), (tree(idx, ws), chosen), (sparse(idx, ws), one), (tree(None, ws), dense)):
                assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert fk.workspace_status(ws) == 0


def test_profile_refuses_no_arrays_and_no_kinds():
    n, ms = (ctypes.c_int32 * 7)(), (ctypes.c_float * 7)()
    for args, word in (((7, None, ms), "null"), ((7, n, None), "null"), ((0, n, ms), "n_kinds"), ((-1, n, ms), "n_kinds")):
        st, msg = _c("fp4kv_profile_read_kinds", *args)
        assert st == 1 and word in msg
    assert _c("fp4kv_profile_read_kinds", 9, (ctypes.c_int32 * 9)(), (ctypes.c_float * 9)())[0] == 0


@gpu
def test_profile_counts_each_operator_by_itself(fk):
    n, H = 900, 64
    packed, scales = make_cache(fk, 1, n, 170)
    x = torch.randn(n, 512, generator=gen(171), device=DEV).bfloat16()
    q = torch.randn(1, 1, H, 512, generator=gen(172), device=DEV).bfloat16()
    lens, mask = torch.tensor([n - 1], dtype=torch.int32, device=DEV), torch.ones(1, 1, dtype=torch.int64, device=DEV)
    short = packed[:, :100].contiguous(), scales[:, :100].contiguous()
    idx = torch.arange(64, dtype=torch.int32, device=DEV).view(1, -1)
    fk.profile_read()
    fk.profile_enable(True)
    try:
        fk.kv_quant_fp4(x, packed[0], scales[0])
        for _ in range(2):
            fk.qkv_norm_rope_fp4(None, x, packed=packed, scales=scales)
        for _ in range(3):
            fk.kv_dequant_fp4(packed, scales)
        fk.sparse_attn_decode(q[:, 0], packed, scales, lens, idx)
        fk.tree_attn_decode(q, packed, scales, lens, mask)           # parts, and the kernel that joins them
        fk.tree_attn_decode(q, *short, lens.clamp(max=99), mask)     # whole items
    finally:
        fk.profile_enable(False)
    got = fk.profile_read()
    counts = {k: c for k, (c, _) in got.items()}
    assert counts == {"kv_quant_fp4": 1, "index_score": 0, "topk_select": 0, "sparse_attn": 1, "qkv_norm_rope_fp4": 2,
                      "kv_dequant_fp4": 3, "tree_attn": 3}, counts
    assert all((ms > 0) == (c > 0) for c, ms in got.values())
    assert all(c == 0 for c, _ in fk.profile_read().values())


@gpu
@pytest.mark.parametrize("B, T, H, cap, every", [(65535, 1, 2, 4, 3), (65535, 2, 1, 3, 1), (4096, 2, 64, 1400, 700)])  # (whole items twice, parts)
def test_tree_batches_of_many_sequences(fk, B, T, H, cap, every):
    """The largest batch, and one in which every 700th sequence alone drafts: against the plain form of all at once.
    Beside what test_tree_rows_that_cancel counts, fp16's least step: a probability's two parts are rounded to
    2^-24 below 2^-14, 2^-25 each, where the row's largest is at least 2^7: 2^-31 sum |v|."""
    g = gen(180)
    packed = torch.randint(0, 256, (B, cap, 256), generator=g, device=DEV).to(torch.uint8)
    scales = torch.randint(0x30, 0x40, (B, cap, 32), generator=g, device=DEV).to(torch.uint8)
    q = torch.randn(B, T, H, 512, generator=g, device=DEV).bfloat16()
    lens = torch.randint(0, cap + 2, (B,), generator=g, device=DEV).int()
    mask = torch.randint(0, 1 << T, (B, T), generator=g, device=DEV)
    drafts = torch.randint(0, T + 1, (B,), generator=g, device=DEV).int()
    drafts[torch.arange(B, device=DEV) % every != every - 1] = 0
    out, lse = torch.full_like(q, 3.0), torch.full((B, T, H), 5.0, device=DEV)
    fk.tree_attn_decode(q, packed, scales, lens, mask, n_draft=drafts, sm_scale=0.04, out=out, lse=lse)
    live = torch.arange(T, device=DEV) < drafts[:, None]
    assert (out[~live] == 3.0).all() and (lse[~live] == 5.0).all()
    rows = drafts.nonzero()[:, 0]
    step = max(1, 30_000 // cap)
    pos = torch.arange(cap, device=DEV)
    for r in rows.split(step):
        v = fk.kv_dequant_fp4(packed[r], scales[r], dtype=torch.float32).view(len(r), cap, 512).double()
        n = lens[r].long().clamp(max=cap)[:, None, None]
        j = pos - n
        see = (j < 0) | ((j < drafts[r].long()[:, None, None]) & ((mask[r][:, :, None] >> j.clamp(0, 63)) & 1 == 1))
        z = torch.einsum("bthc,bnc->bthn", q[r].double(), v) * float(np.float32(0.04))
        dz = 2.0 ** -16 * 0.04 * torch.einsum("bthc,bnc->bthn", q[r].double().abs(), v.abs()).amax(-1, keepdim=True)
        z = z.masked_fill(~see[:, :, None], -np.inf)
        want_l = torch.logsumexp(z, -1)
        p = torch.exp(z - want_l[..., None]).nan_to_num(0.0)  # (a token that sees nothing)
        want, A = torch.einsum("bthn,bnc->bthc", p, v), torch.einsum("bthn,bnc->bthc", p, v.abs())
        ok = live[r]
        least = 2.0 ** -31 * v.abs().sum(1)[:, None, None]
        off = (out[r].double() - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -16 + 2 * dz) * A + least)
        assert (off[ok] <= 0).all()
        inf = torch.isneginf(want_l)
        assert torch.equal(torch.isneginf(lse[r])[ok], inf[ok])
        assert ((lse[r].double() - want_l).abs() <= dz[..., 0] + 2.0 ** -20 * (1 + want_l.abs()))[ok[..., None] & ~inf].all()
