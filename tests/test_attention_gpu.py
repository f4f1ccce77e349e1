"""Cross attention and prefix attention against plain attention in 64 bits, element by
element, with the bounds that attention_util derives from the kernels' roundings."""
import math

import pytest
import torch

import attention_util as au

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def att():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_memory_attention_b200 import attention
    return attention


def lens(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32, device="cuda")


def cross_inputs(B, Hq, Hkv, n, m, d, dtype, layout="bhnd", seed=0):
    q = au.randn((B, Hq, n, d), dtype, seed + 1, layout, 2.0)
    k = au.randn((B, Hkv, m, d), dtype, seed + 2, layout)
    v = au.randn((B, Hkv, m, d), dtype, seed + 3, layout)
    do = au.randn((B, Hq, n, d), dtype, seed + 4, layout)
    return q, k, v, do, 1.0 / math.sqrt(d)


# (B, Hq, Hkv, n, m, k_len): one key, one row, tiles and their neighbours, grouped heads,
# empty, short and out-of-range lengths.
CROSS = [
    (1, 1, 1, 1, 1, None),
    (1, 2, 1, 1, 65, None),
    (2, 4, 2, 3, 64, [64, 0]),
    (1, 3, 3, 64, 63, None),
    (1, 2, 2, 65, 128, None),
    (3, 2, 1, 127, 129, [129, 1, 0]),
    (1, 2, 2, 129, 255, None),
    (2, 8, 2, 40, 257, [-5, 1000]),
    (2, 1, 1, 300, 517, [511, 128]),
    (1, 8, 1, 1, 900, [333]),
    (5, 6, 3, 2, 130, [0, 130, 127, 129, 64]),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CROSS, ids=lambda c: "x".join(map(str, c[:5])))
def test_cross_attention(att, case, dtype, d):
    B, Hq, Hkv, n, m, k_len = case
    q, k, v, do, tau = cross_inputs(B, Hq, Hkv, n, m, d, dtype, seed=d + n)
    got = att.cross_attention(q, k, v, tau, lens(k_len), dout=do)
    att.lard_attn_device_status()
    au.check(got, au.cross(q, k, v, tau, k_len, do))


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["bnhd", "wide"])
def test_strided_inputs_and_outputs(att, layout, dtype):
    """Views in, views out; what lies around an output view is left as it was."""
    B, Hq, Hkv, n, m, d = 2, 4, 2, 70, 150, 64
    q, k, v, do, tau = cross_inputs(B, Hq, Hkv, n, m, d, dtype, layout, seed=5)
    want = au.cross(q, k, v, tau, [150, 77], do)
    k_len, size = lens([150, 77]), {"q": (B, Hq, n, d), "k": (B, Hkv, m, d)}
    got = {}
    around = {}
    for name, like in (("out", "q"), ("dq", "q"), ("dk", "k"), ("dv", "k")):
        t = au.randn(size[like], dtype, 9, layout)
        got[name] = t.fill_(7.0)
        around[name] = t._base.clone() if layout == "wide" else None
    got["lse"] = torch.empty((B, Hq, n), device="cuda")
    ws = torch.full((max(att.lard_cross_attn_fwd_workspace_bytes(q, k),
                         att.lard_cross_attn_bwd_workspace_bytes(q, k), 16),), 255, dtype=torch.uint8, device="cuda")
    att.lard_cross_attn_fwd(q, k, v, tau, got["out"], got["lse"], k_len, ws)
    ws.fill_(255)  # NaN in every type
    att.lard_cross_attn_bwd(q, k, v, tau, got["out"], got["lse"], do, got["dq"], got["dk"], got["dv"], k_len, ws)
    au.check(got, want)
    for name, before in around.items():
        if before is not None:
            after = got[name]._base.clone()
            after[:B, 1:-1, 2:-1, 8:-8] = before[:B, 1:-1, 2:-1, 8:-8]
            assert torch.equal(after.nan_to_num(3.0), before.nan_to_num(3.0)), name


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 40, 200])
def test_padding_may_hold_anything(att, n, dtype):
    """Infinities and NaN in key and value rows past the length reach nothing."""
    q, k, v, do, tau = cross_inputs(2, 4, 2, n, 333, 64, dtype, seed=11)
    k_len = [200, 65]
    want = au.cross(q, k, v, tau, k_len, do)
    for b, size in enumerate(k_len):
        k[b, :, size:] = float("nan")
        v[b, :, size::2] = float("inf")
        v[b, :, size + 1::2] = float("nan")
    au.check(att.cross_attention(q, k, v, tau, lens(k_len), dout=do), want)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,m", [(40, 150), (4, 2000)])
def test_gradient_rows_past_the_length_are_zeros(att, n, m, dtype):
    """Also where the upstream gradient holds infinities and NaN."""
    q, k, v, do, tau = cross_inputs(2, 4, 2, n, m, 64, dtype, seed=15)
    k_len = [70, 0]
    do[:, :, 0] = float("inf")
    do[:, :, n - 1] = float("nan")
    got = att.cross_attention(q, k, v, tau, lens(k_len), dout=do)
    for b, size in enumerate(k_len):
        assert not got["dk"][b, :, size:].any() and not got["dv"][b, :, size:].any()
    assert not got["dq"][1].any() and not got["out"][1].any()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [130, 16])
def test_offsets_past_32_bits(att, n, dtype):
    """Rows, heads and tensors of one buffer of more than 2^31 elements, eight views interleaved."""
    B, H, d, step = 1, 2, 64, 1 << 24
    big = torch.empty(((n if n > 128 else 130) * step,), dtype=dtype, device="cuda")
    row = step if n > 128 else 2 * d * 8
    head = d * 8 if n > 128 else 1 << 31
    at = {}
    for x, name in enumerate(("q", "k", "v", "do", "out", "dq", "dk", "dv")):
        at[name] = big.as_strided((B, H, n, d), (0, head, row, 1), x * d)
        at[name].copy_(au.randn((B, H, n, d), dtype, 170 + x))
    q, k, v, do, tau = at["q"], at["k"], at["v"], at["do"], 1.0 / math.sqrt(d)
    want = au.cross(q, k, v, tau, None, do)
    at["lse"] = torch.empty((B, H, n), device="cuda")
    ws = torch.empty((max(att.lard_cross_attn_fwd_workspace_bytes(q, k),
                          att.lard_cross_attn_bwd_workspace_bytes(q, k), 16),), dtype=torch.uint8, device="cuda")
    att.lard_cross_attn_fwd(q, k, v, tau, at["out"], at["lse"], None, ws)
    att.lard_cross_attn_bwd(q, k, v, tau, at["out"], at["lse"], do, at["dq"], at["dk"], at["dv"], None, ws)
    att.lard_attn_device_status()
    au.check(at, want)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [3, 60, 460])
def test_many_rows_that_see_no_key(att, n, d, dtype):
    """Every row of every head of an empty sequence: zeros and -infinity, beside ones that see some keys."""
    q, k, v, do, tau = cross_inputs(6, 32, 2, n, 16, d, dtype, "bnhd", seed=17)
    k_len = [14, -1, 0, 15, 0, 0]
    got = att.cross_attention(q, k, v, tau, lens(k_len), dout=do)
    for b in (1, 2, 4, 5):
        assert not got["out"][b].any() and (got["lse"][b] == -math.inf).all()
        assert not got["dq"][b].any() and not got["dk"][b].any() and not got["dv"][b].any()
    assert got["out"][0].any() and got["dq"][3].any()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_shared_keys(att, dtype):
    """One key block for all sequences (batch stride 0) and for all heads (head stride 0)."""
    q, k, v, _, tau = cross_inputs(3, 4, 2, 33, 90, 64, dtype, seed=21)
    kb, vh = k[:1].expand(3, 2, 90, 64), v[:, :1].expand(3, 2, 90, 64)
    au.check(att.cross_attention(q, kb, vh, tau), au.cross(q, kb, vh, tau))


@pytest.mark.parametrize("n,m", [(1, 5000), (3, 2500), (20, 4001)])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_few_rows_over_many_keys(att, n, m, dtype):
    """The key axis is split over blocks and joined; some splits see nothing."""
    q, k, v, _, tau = cross_inputs(2, 4, 1, n, m, 128, dtype, seed=31)
    k_len = [m, 17]
    au.check(att.cross_attention(q, k, v, tau, lens(k_len)), au.cross(q, k, v, tau, k_len))


@pytest.mark.parametrize("n,m", [(3, 3000), (700, 40), (130, 400), (1, 257)])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
def test_gradients_of_long_and_narrow_calls(att, n, m, dtype, d):
    """Few blocks along one axis: the other is split and its partial sums are added; some
    splits have nothing to do."""
    q, k, v, do, tau = cross_inputs(2, 4, 2, n, m, d, dtype, seed=35)
    k_len = [m, 30]
    got = att.cross_attention(q, k, v, tau, lens(k_len), dout=do)
    att.lard_attn_device_status()
    au.check(got, au.cross(q, k, v, tau, k_len, do))


# One row tile and several, few rows, and both with the key axis split.
@pytest.mark.parametrize("n,m", [(3, 90), (2, 9000), (30, 200), (40, 4000), (300, 260), (300, 3000)])
@pytest.mark.parametrize("d", [64, 128])
def test_rest_of_the_rounding(att, n, m, d):
    """out + rest is the output to twice the digits, whichever kernel wrote them, and the
    gradients that take both have no part of out's rounding in delta."""
    q, k, v, do, tau = cross_inputs(2, 4, 2, n, m, d, BF16, "bnhd", seed=37)
    k_len = [m, m // 2]
    got = {x: torch.empty_like(q) for x in ("out", "rest", "dq")} | {x: torch.empty_like(k) for x in ("dk", "dv")}
    got["lse"] = torch.empty((2, 4, n), device="cuda")
    ws = torch.empty((max(att.lard_cross_attn_fwd_workspace_bytes(q, k),
                          att.lard_cross_attn_bwd_workspace_bytes(q, k)),), dtype=torch.uint8, device="cuda")
    att.lard_cross_attn_fwd(q, k, v, tau, got["out"], got["lse"], lens(k_len), ws, rest=got["rest"])
    att.lard_cross_attn_bwd(q, k, v, tau, got["out"], got["lse"], do, got["dq"], got["dk"], got["dv"], lens(k_len), ws,
                            rest=got["rest"])
    att.lard_attn_device_status()
    got["sum"] = got["out"].double() + got["rest"].double()
    au.check(got, au.cross(q, k, v, tau, k_len, do, rest=True))


def test_large_and_rising_logits(att):
    """Row maxima that rise tile after tile by far, and logits of several hundreds."""
    for dtype in (BF16, FP32):
        q, k, v, do, _ = cross_inputs(1, 2, 2, 140, 700, 64, dtype, seed=41)
        k = (k * torch.linspace(0.1, 9.0, 700, device="cuda")[:, None]).to(dtype)
        au.check(att.cross_attention(q, k, v, 0.5), au.cross(q, k, v, 0.5))
        k = k.flip(2).contiguous()
        au.check(att.cross_attention(q, k, v, 0.5), au.cross(q, k, v, 0.5))


# (B, Hq, Hkv, n, P, S, s_len)
PREFIX = [
    (1, 1, 1, 1, 1, 1, None),
    (4, 4, 2, 1, 200, 70, [70, 1, 33, 64]),
    (2, 8, 2, 3, 129, 20, [20, 3]),
    (3, 4, 4, 5, 64, 40, [2, 0, 5]),       # fewer rows of their own than new ones
    (2, 4, 1, 70, 300, 200, [200, 130]),
    (2, 2, 2, 130, 65, 140, [135, 140]),
    (3, 4, 2, 2, 0, 90, [90, 0, 65]),      # no shared prefix
    (3, 4, 2, 2, 500, 0, None),            # nothing of their own
    (2, 2, 1, 4, 257, 128, [-3, 9999]),
    (17, 8, 1, 1, 3000, 30, None),
]


def prefix_inputs(B, Hq, Hkv, n, P, S, d, dtype, layout="bhnd", seed=0):
    q = au.randn((B, Hq, n, d), dtype, seed + 1, layout, 2.0)
    kp, vp = ((au.randn((1, Hkv, P, d), dtype, seed + s, layout)[0] if P else None) for s in (2, 3))
    ks, vs = ((au.randn((B, Hkv, S, d), dtype, seed + s, layout) if S else None) for s in (4, 5))
    return q, kp, vp, ks, vs, 1.0 / math.sqrt(d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "x".join(map(str, c[:6])))
def test_prefix_attention(att, case, dtype, d):
    B, Hq, Hkv, n, P, S, s_len = case
    layout = ["bhnd", "bnhd", "wide"][(n + P) % 3]
    q, kp, vp, ks, vs, tau = prefix_inputs(B, Hq, Hkv, n, P, S, d, dtype, layout, seed=d + n)
    got = att.prefix_attention(q, kp, vp, ks, vs, lens(s_len), tau)
    att.lard_attn_device_status()
    au.check(got, au.prefix(q, kp, vp, ks, vs, s_len, tau))


# One sequence takes shared and own rows in one pass: both may end inside a tile.
ONE = [(1, 4, 2, 3, 239, 60), (1, 2, 1, 40, 15, 2), (1, 4, 2, 67, 2, 99), (1, 2, 2, 5, 242, 9),
       (1, 2, 1, 174, 8, 12), (1, 2, 2, 19, 754, 118), (1, 2, 1, 300, 2000, 301), (1, 16, 1, 1, 1000, 31)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", ONE, ids=lambda c: "x".join(map(str, c)))
def test_prefix_of_one_sequence(att, case, dtype, d):
    B, Hq, Hkv, n, P, S = case
    for s_len in (None, [S // 2]):
        q, kp, vp, ks, vs, tau = prefix_inputs(B, Hq, Hkv, n, P, S, d, dtype, seed=d + n)
        got = att.prefix_attention(q, kp, vp, ks, vs, lens(s_len), tau)
        att.lard_attn_device_status()
        au.check(got, au.prefix(q, kp, vp, ks, vs, s_len, tau))


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_prefix_padding_may_hold_anything(att, dtype):
    q, kp, vp, ks, vs, tau = prefix_inputs(3, 4, 2, 2, 150, 100, 128, dtype, seed=3)
    s_len = [100, 40, 0]
    want = au.prefix(q, kp, vp, ks, vs, s_len, tau)
    for b, size in enumerate(s_len):
        ks[b, :, size:] = float("inf")
        vs[b, :, size:] = float("nan")
    au.check(att.prefix_attention(q, kp, vp, ks, vs, lens(s_len), tau), want)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_a_training_step_and_then_decoding(att, dtype):
    """The operators as they are used together: a layer's cross attention and its gradients;
    then the same rows one at a time, which give the same outputs; then the encoded states as
    a prefix that a batch of sequences shares."""
    B, Hq, Hkv, n, m, d = 2, 8, 2, 37, 290, 64
    q, k, v, do, tau = cross_inputs(B, Hq, Hkv, n, m, d, dtype, "bnhd", seed=61)
    k_len = [290, 123]
    want = au.cross(q, k, v, tau, k_len, do)
    au.check(att.cross_attention(q, k, v, tau, lens(k_len), dout=do), want)
    for i in (0, 17, n - 1):
        one = att.cross_attention(q[:, :, i:i + 1], k, v, tau, lens(k_len))
        au.check(one, {x: (want[x][0][:, :, i:i + 1], want[x][1][:, :, i:i + 1]) for x in ("out", "lse")})
    kp, vp = k[0], v[0]
    shared = att.prefix_attention(q, kp, vp, None, None, None, tau)
    au.check(shared, au.cross(q, k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1), tau))
    own = att.prefix_attention(q[:, :, :1], kp, vp, k, v, lens(k_len), tau)
    au.check(own, au.prefix(q[:, :, :1], kp, vp, k, v, k_len, tau))


def test_gradients_against_differences(att):
    """Directional derivatives of L = sum(dO * O), by central differences of the 64-bit
    forward pass: h = 2^-12 leaves h^2 times the third derivative (some units here, 6e-8
    of the directions' norms) and 2^-52 / h; the fp32 gradients bring their own bound."""
    q, k, v, do, tau = cross_inputs(2, 4, 2, 9, 21, 64, FP32, seed=71)
    k_len = [21, 13]
    got = att.cross_attention(q, k, v, tau, lens(k_len), dout=do)
    bound = au.cross(q, k, v, tau, k_len, do)
    x = {"q": au.f64(q), "k": au.f64(k), "v": au.f64(v)}

    def loss(q, k, v):
        total = 0.0
        for b in range(2):
            for h in range(4):
                kk, vv = k[b, h // 2, :k_len[b]], v[b, h // 2, :k_len[b]]
                total += (torch.softmax(tau * q[b, h] @ kk.T, -1) @ vv * au.f64(do)[b, h]).sum()
        return total

    gen = torch.Generator().manual_seed(1)
    for name in x:
        for _ in range(3):
            way = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
            h = 2.0 ** -12
            plus, minus = dict(x), dict(x)
            plus[name], minus[name] = x[name] + h * way, x[name] - h * way
            diff = (loss(**plus) - loss(**minus)) / (2 * h)
            mine = (au.f64(got["d" + name]) * way).sum()
            room = (bound["d" + name][1] * way.abs()).sum() + 1e-6 * way.norm() * au.f64(do).norm()
            assert abs(mine - diff) <= room, (name, mine.item(), diff.item(), room.item())


def test_forward_is_deterministic(att):
    for n, m in ((1, 3001), (500, 700)):
        for dtype in (BF16, FP32):
            q, k, v, _, tau = cross_inputs(2, 4, 2, n, m, 128, dtype, seed=81)
            first = att.cross_attention(q, k, v, tau)
            for _ in range(3):
                again = att.cross_attention(q, k, v, tau)
                assert torch.equal(first["out"], again["out"]) and torch.equal(first["lse"], again["lse"])


class Guarded:
    """Buffers with guard bytes on either side of each."""

    def __init__(self):
        self.all = []

    def empty(self, shape, dtype):
        size = math.prod(shape) * dtype.itemsize
        raw = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((raw, size))
        return raw[256:256 + size].view(dtype).view(shape)

    def check(self):
        for raw, size in self.all:
            assert (raw[:256] == 0xA5).all() and (raw[256 + size:] == 0xA5).all()


def parts(need, rows, d):
    """Parts of each row that a forward call of this workspace joins."""
    return need // (rows * (4 * d + 4))


# From 8192 rows on a warp joins eight rows; neither count is a multiple of eight.
# (B, Hq, Hkv, n, P, S): two parts a row; nine (five at d = 128 in bf16), which four lanes share.
@pytest.mark.parametrize("case", [(3, 7, 7, 391, 70, 50), (51, 7, 1, 23, 3000, 30)], ids=["two parts", "many parts"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_join_of_many_rows(att, case, dtype, d):
    B, Hq, Hkv, n, P, S = case
    q, kp, vp, ks, vs, tau = prefix_inputs(B, Hq, Hkv, n, P, S, d, dtype, "bnhd", seed=d + P)
    s_len = [(S + 7 * b) % (S + 1) for b in range(B)]
    need = att.lard_prefix_attn_workspace_bytes(q, kp, ks)
    assert B * Hq * n > 8192 and B * Hq * n % 8 and (parts(need, B * Hq * n, d) == 2) == (P == 70)
    guard = Guarded()
    got = {"out": guard.empty(q.shape, dtype), "lse": guard.empty((B, Hq, n), FP32)}
    att.lard_prefix_attn(q, kp, vp, ks, vs, lens(s_len), tau, got["out"], got["lse"], guard.empty((need,), torch.uint8))
    att.lard_attn_device_status()
    au.check(got, au.prefix(q, kp, vp, ks, vs, s_len, tau))
    guard.check()


@pytest.mark.parametrize("dtype,m", [(BF16, 1000), (FP32, 3000)], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [900, 30, 0])
def test_join_of_many_rows_with_rest(att, dtype, m, d, size):
    """The same join of one long sequence's rows, with what rounding leaves of them; of the shorter
    lengths most parts, or all, have seen nothing."""
    n = 8203
    q, k, v, _, tau = cross_inputs(1, 1, 1, n, m, d, dtype, seed=181)
    need = att.lard_cross_attn_fwd_workspace_bytes(q, k)
    assert parts(need, n, d) >= 4
    guard = Guarded()
    got = {"out": guard.empty(q.shape, dtype), "lse": guard.empty((1, 1, n), FP32)}
    if dtype is BF16:
        got["rest"] = guard.empty(q.shape, dtype)
    att.lard_cross_attn_fwd(q, k, v, tau, got["out"], got["lse"], lens([size]), guard.empty((need,), torch.uint8),
                            rest=got.get("rest"))
    att.lard_attn_device_status()
    if dtype is BF16:
        got["sum"] = got["out"].double() + got["rest"].double()
    au.check(got, au.cross(q, k, v, tau, [size], rest=dtype is BF16))
    guard.check()


# Few problems of many keys: several clusters of blocks share a problem's keys in bf16.
@pytest.mark.parametrize("case", [(2, 8, 2, 1, 17000, [17000, 40]), (1, 8, 1, 2, 40000, [39999]),
                                  (1, 4, 1, 4, 40000, [21]), (4, 4, 1, 3, 20000, [20000, 0, 333, 9001])],
                         ids=lambda c: "x".join(map(str, c[:5])))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_few_rows_over_very_many_keys(att, case, dtype, d):
    B, Hq, Hkv, n, m, k_len = case
    q, k, v, _, tau = cross_inputs(B, Hq, Hkv, n, m, d, dtype, "bnhd", seed=191)
    need = att.lard_cross_attn_fwd_workspace_bytes(q, k)
    assert parts(need, B * Hq * n, d) >= 2
    guard = Guarded()
    got = {"out": guard.empty(q.shape, dtype), "lse": guard.empty((B, Hq, n), FP32)}
    if dtype is BF16:
        got["rest"] = guard.empty(q.shape, dtype)
    att.lard_cross_attn_fwd(q, k, v, tau, got["out"], got["lse"], lens(k_len), guard.empty((need,), torch.uint8),
                            rest=got.get("rest"))
    att.lard_attn_device_status()
    au.check(got, au.cross(q, k, v, tau, k_len))
    guard.check()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_one_token_behind_a_very_long_prefix(att, dtype):
    """The clusters' runs of keys pass from the shared rows to the sequence's own."""
    for P, S, s_len in ((20001, 77, [50]), (13, 20000, [19990])):
        q, kp, vp, ks, vs, tau = prefix_inputs(1, 8, 2, 2, P, S, 128, dtype, seed=195)
        assert parts(att.lard_prefix_attn_workspace_bytes(q, kp, ks), 16, 128) >= 2
        got = att.prefix_attention(q, kp, vp, ks, vs, lens(s_len), tau)
        att.lard_attn_device_status()
        au.check(got, au.prefix(q, kp, vp, ks, vs, s_len, tau))


# Both axes split, one of them, neither (bf16); each with an empty tail.
@pytest.mark.parametrize("B,Hq,Hkv,n,m", [(1, 4, 2, 200, 900), (1, 4, 2, 5, 7000), (4, 10, 10, 500, 520)])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_gradients_repeat_bit_for_bit(att, B, Hq, Hkv, n, m, dtype):
    q, k, v, do, tau = cross_inputs(B, Hq, Hkv, n, m, 128, dtype, "bnhd", seed=201)
    k_len = lens([m - 30 * (b + 1) for b in range(B)])
    first = att.cross_attention(q, k, v, tau, k_len, dout=do)
    for _ in range(4):
        again = att.cross_attention(q, k, v, tau, k_len, dout=do)
        for name in first:
            assert torch.equal(first[name], again[name]), name
    assert first["dq"].any() and first["dk"].any() and first["dv"].any()


@pytest.mark.parametrize("n", [6, 150])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_gradients_of_shared_inputs(att, n, dtype):
    """Queries and upstream gradients shared by all heads, keys by all sequences, values by all
    key heads (strides of 0): the gradients are those of every sequence and head."""
    B, Hq, Hkv, m, d = 3, 4, 2, 140, 64
    q, k, v, do, tau = cross_inputs(B, Hq, Hkv, n, m, d, dtype, seed=211)
    q, do = q[:, :1].expand(B, Hq, n, d), do[:1, :1].expand(B, Hq, n, d)
    k, v = k[:1].expand(B, Hkv, m, d), v[:, :1].expand(B, Hkv, m, d)
    got = att.cross_attention(q, k, v, tau, lens([140, 0, 77]), dout=do)
    att.lard_attn_device_status()
    au.check(got, au.cross(q, k, v, tau, [140, 0, 77], do))


def test_captured_calls_replay_with_other_lengths(att):
    """Forward, backward and prefix calls in one graph; replays follow the lengths and inputs
    in device memory.  An eager call in between uses memory of its own."""
    q, k, v, do, tau = cross_inputs(2, 4, 2, 30, 260, 64, BF16, seed=91)
    qd, kp, vp, ks, vs, _ = prefix_inputs(2, 4, 2, 1, 600, 50, 64, BF16, seed=92)
    k_len, s_len = lens([260, 100]), lens([50, 7])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # first use outside of the capture
        att.cross_attention(q, k, v, tau, k_len, dout=do)
        att.prefix_attention(qd, kp, vp, ks, vs, s_len, tau)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train = att.cross_attention(q, k, v, tau, k_len, dout=do)
        token = att.prefix_attention(qd, kp, vp, ks, vs, s_len, tau)
    for a, b in (([260, 100], [50, 7]), ([0, 260], [1, 50]), ([129, 1], [20, 0])):
        k_len.copy_(torch.tensor(a, dtype=torch.int32))
        s_len.copy_(torch.tensor(b, dtype=torch.int32))
        graph.replay()
        eager = att.cross_attention(q, k, v, tau, k_len, dout=do)
        torch.cuda.synchronize()
        want = au.cross(q, k, v, tau, a, do)
        au.check(train, want, "replayed")
        au.check(eager, want, "eager")
        au.check(token, au.prefix(qd, kp, vp, ks, vs, b, tau), "replayed")
    att.lard_attn_device_status()


def test_two_streams_at_once(att):
    """Calls on two streams, each with what it allocates on its own stream."""
    cases = [cross_inputs(2, 8, 2, 1, 4000, 128, BF16, seed=s) for s in (101, 111)]
    cases += [cross_inputs(1, 4, 4, 200, 500, 64, BF16, seed=s) for s in (121, 131)]
    want = [au.cross(q, k, v, tau, None, do) for q, k, v, do, tau in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [att.cross_attention(q, k, v, tau, dout=do, stream=streams[i % 2])
               for i, (q, k, v, do, tau) in enumerate(cases)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        au.check(g, w)
    for s in streams:
        att.lard_attn_device_status(s)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_calls_follow_the_given_stream(att, raw):
    """Inputs that the given stream is still to write, behind some 50 ms of other work, while the
    current stream is idle: the calls come after them."""
    q, k, v, do, tau = cross_inputs(2, 4, 2, 33, 170, 64, BF16, seed=161)
    late = [torch.zeros_like(x) for x in (q, k, v, do)]
    side = torch.cuda.Stream()
    given = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        for x, y in zip(late, (q, k, v, do)):
            x.copy_(y)
    got = att.cross_attention(*late[:3], tau, dout=late[3], stream=given)
    shared = att.prefix_attention(late[0], late[1][0], late[2][0], None, None, None, tau, stream=given)
    assert torch.cuda.current_stream() != side
    att.lard_attn_device_status(given)
    au.check(got, au.cross(q, k, v, tau, None, do))
    au.check(shared, au.cross(q, k[:1].expand(2, -1, -1, -1), v[:1].expand(2, -1, -1, -1), tau))


def test_interleaved_outputs(att):
    """dK and dV as the two halves of one [B, m, 2, H, d] buffer, as a fused projection has it."""
    q, k, v, do, tau = cross_inputs(2, 4, 2, 20, 90, 64, BF16, seed=141)
    got = att.cross_attention(q, k, v, tau)
    both = torch.zeros((2, 90, 2, 2, 64), dtype=BF16, device="cuda")
    got["dk"], got["dv"], got["dq"] = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2), torch.empty_like(q)
    ws = torch.empty((att.lard_cross_attn_bwd_workspace_bytes(q, k),), dtype=torch.uint8, device="cuda")
    att.lard_cross_attn_bwd(q, k, v, tau, got["out"], got["lse"], do, got["dq"], got["dk"], got["dv"], None, ws)
    au.check(got, au.cross(q, k, v, tau, None, do))


def test_host_buffers_are_refused(att):
    """A pointer that is not device memory is refused by the library before any launch."""
    q, k, v, _, tau = cross_inputs(1, 1, 1, 4, 8, 64, BF16, seed=151)
    out, lse = torch.empty_like(q), torch.empty((1, 1, 4), device="cuda")
    host = torch.empty((1, 1, 8, 64), dtype=BF16).pin_memory()
    args = list(att._CROSS.unpack(att._cross_args(q, k, v, tau, None, out, lse)))
    args[12] = host.data_ptr()  # k
    st = att._lib.lard_cross_attn_fwd(att._CROSS.pack(*args), None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 1
    with pytest.raises(ValueError):
        att.cross_attention(q, host, host, tau)
