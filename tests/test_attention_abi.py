"""CPU checks of the attention library's C ABI: it exports what include/lard_attn.h declares
and refuses bad arguments before any CUDA call (the addresses below are made up)."""
import contextlib
import ctypes
import os
import re
import subprocess
import sys
import types

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lard_attn.h")


class View(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("batch", ctypes.c_longlong), ("head", ctypes.c_longlong),
                ("row", ctypes.c_longlong)]


class Cross(ctypes.Structure):
    _fields_ = ([(x, ctypes.c_int) for x in ("dtype", "B", "Hq", "Hkv", "n", "m", "d")] + [("tau", ctypes.c_float)] +
                [(x, View) for x in "qkv"] + [("k_len", ctypes.c_void_p), ("out", View), ("lse", ctypes.c_void_p)] +
                [(x, View) for x in ("dout", "dq", "dk", "dv", "rest")])


class Prefix(ctypes.Structure):
    _fields_ = ([(x, ctypes.c_int) for x in ("dtype", "B", "Hq", "Hkv", "n", "P", "S", "d")] + [("tau", ctypes.c_float)] +
                [(x, View) for x in ("q", "kp", "vp", "ks", "vs")] +
                [("s_len", ctypes.c_void_p), ("out", View), ("lse", ctypes.c_void_p)])


@pytest.fixture(scope="module")
def att():
    from linear_memory_attention_b200 import build
    build.build()
    from linear_memory_attention_b200 import attention
    return attention


def test_exports_match_the_header(att):
    text = open(HEADER).read()
    names = re.findall(r"LARD_API\s+[\w\s\*]+?\b(lard_\w+)\s*\(", text)
    assert set(names) == set(att.EXPORTS) and len(names) == len(set(names))
    for name in names:
        assert hasattr(att._lib, name)


def test_packed_arguments_have_the_structs_layout(att):
    assert att._CROSS.size == ctypes.sizeof(Cross) and att._PREFIX.size == ctypes.sizeof(Prefix)
    c = Cross.from_buffer_copy(att._CROSS.pack(*range(7), 0.5, *range(8, 46)))
    assert (c.d, c.tau, c.q.ptr, c.k.ptr, c.v.row, c.k_len, c.out.ptr, c.lse, c.dout.ptr, c.dv.row, c.rest.ptr) == (
        6, 0.5, 8, 12, 19, 20, 21, 25, 26, 41, 42)
    p = Prefix.from_buffer_copy(att._PREFIX.pack(*range(8), 0.5, *range(9, 35)))
    assert (p.d, p.tau, p.q.ptr, p.kp.ptr, p.vs.row, p.s_len, p.out.ptr, p.lse) == (7, 0.5, 9, 13, 28, 29, 30, 34)


def view(ptr, H, rows, d):
    return View(ptr, H * rows * d, rows * d, d)


STEP = 0x1000000  # more than any tensor here


def cross_call(att, fn="fwd", ws=40 * STEP, ws_bytes=None, **kw):
    """An in-order call on made-up addresses, changed by kw; returns the status."""
    B, Hq, Hkv, n, m, d = (kw.pop(x, y) for x, y in (("B", 2), ("Hq", 4), ("Hkv", 2), ("n", 50), ("m", 70), ("d", 64)))
    a = Cross(dtype=kw.pop("dtype", 0), B=B, Hq=Hq, Hkv=Hkv, n=n, m=m, d=d, tau=kw.pop("tau", 0.1), k_len=20 * STEP,
              lse=21 * STEP)
    for i, (x, H, rows) in enumerate((("q", Hq, n), ("k", Hkv, m), ("v", Hkv, m), ("out", Hq, n), ("dout", Hq, n),
                                      ("dq", Hq, n), ("dk", Hkv, m), ("dv", Hkv, m))):
        setattr(a, x, view((i + 1) * STEP, H, rows, d))
    for x, y in kw.items():
        if "_" in x and x != "k_len":
            name, part = x.split("_")
            setattr(getattr(a, name), part, y)
        else:
            setattr(a, x, y)
    size = getattr(att._lib, f"lard_cross_attn_{fn}_workspace_bytes")(ctypes.byref(a))
    return getattr(att._lib, f"lard_cross_attn_{fn}")(ctypes.byref(a), ws, size if ws_bytes is None else ws_bytes, None)


def test_valid_arguments_reach_the_device_check(att):
    """Without a GPU the calls below end there with LARD_ERR_CUDA, so that the refusals (1, 2)
    are those of the argument checks; with one, the made-up addresses are refused there."""
    end = 1 if torch.cuda.is_available() else 3
    assert cross_call(att) == end and cross_call(att, "bwd") == end and prefix_call(att) == end
    assert prefix_call(att, P=100000) == end
    assert cross_call(att, k_batch=0, v_head=0) == end                 # inputs may be shared
    rest = dict(rest_ptr=9 * STEP, rest_batch=4 * 50 * 64, rest_head=50 * 64, rest_row=64)
    assert cross_call(att, **rest) == end and cross_call(att, "bwd", **rest) == end
    assert cross_call(att, **dict(rest, rest_ptr=4 * STEP)) == 1 and cross_call(att, **dict(rest, rest_row=63)) == 1
    assert cross_call(att, "bwd", **dict(rest, rest_ptr=6 * STEP)) == 1     # an input of the backward pass, over dq
    assert cross_call(att, dtype=1, **dict(rest, rest_ptr=4 * STEP)) == end  # not used for fp32
    assert cross_call(att, B=1, q_batch=7, out_batch=3) == end         # the stride of one element is not used
    assert prefix_call(att, P=0, kp_ptr=None, vp_ptr=None) == end
    assert prefix_call(att, S=0, ks_ptr=None, vs_ptr=None, s_len=1) == end
    # dK and dV as the halves of one [B, m, 2, Hkv, d] buffer
    halves = dict(dk_batch=70 * 256, dk_row=256, dk_head=64, dv_ptr=7 * STEP + 256, dv_batch=70 * 256, dv_row=256,
                  dv_head=64)
    assert cross_call(att, "bwd", **halves) == end
    assert cross_call(att, "bwd", **dict(halves, dv_ptr=7 * STEP + 128)) == 1   # one head of each overlaps


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(n=0), dict(m=0), dict(Hq=3), dict(Hkv=0), dict(tau=0.0), dict(tau=float("nan")),
    dict(tau=float("inf")), dict(n=2 ** 31 - 1), dict(m=2 ** 31 - 1), dict(B=1 << 20, Hq=1 << 12), dict(q_ptr=None),
    dict(k_ptr=2 * STEP + 8), dict(lse=None), dict(lse=21 * STEP + 2), dict(k_len=20 * STEP + 1), dict(q_row=66),
    dict(q_row=32), dict(v_head=-64), dict(out_head=0), dict(out_batch=64), dict(out_row=60), dict(out_ptr=STEP),
    dict(lse=STEP), dict(lse=4 * STEP), dict(k_len=21 * STEP), dict(q_batch=1 << 40),
])
def test_forward_refuses(att, kw):
    assert cross_call(att, **kw) == 1


@pytest.mark.parametrize("kw", [dict(d=32), dict(d=96), dict(d=256), dict(dtype=2), dict(dtype=-1)])
def test_unsupported_types_and_head_sizes(att, kw):
    assert cross_call(att, **kw) == 2 and cross_call(att, "bwd", **kw) == 2 and prefix_call(att, **kw) == 2


@pytest.mark.parametrize("kw", [
    dict(dq_ptr=None), dict(dk_ptr=8 * STEP), dict(dv_ptr=7 * STEP + 16), dict(dq_ptr=5 * STEP), dict(dout_ptr=None),
    dict(dk_head=0), dict(out_ptr=None), dict(dv_ptr=2 * STEP), dict(lse=6 * STEP), dict(ws=40 * STEP + 4),
    dict(ws=None), dict(ws_bytes=8), dict(ws=6 * STEP),
])
def test_backward_refuses(att, kw):
    assert cross_call(att, "bwd", **kw) == 1


def prefix_call(att, ws=40 * STEP, **kw):
    B, Hq, Hkv, n, P, S, d = (kw.pop(x, y) for x, y in (("B", 2), ("Hq", 4), ("Hkv", 2), ("n", 3), ("P", 900), ("S", 70),
                                                       ("d", 64)))
    a = Prefix(dtype=kw.pop("dtype", 0), B=B, Hq=Hq, Hkv=Hkv, n=n, P=P, S=S, d=d, tau=kw.pop("tau", 0.1),
               s_len=20 * STEP, lse=21 * STEP)
    for i, (x, H, rows) in enumerate((("q", Hq, n), ("kp", Hkv, P), ("vp", Hkv, P), ("ks", Hkv, S), ("vs", Hkv, S),
                                      ("out", Hq, n))):
        setattr(a, x, view((i + 1) * STEP, H, rows, d))
    for x, y in kw.items():
        if "_" in x and x != "s_len":
            name, part = x.split("_")
            setattr(getattr(a, name), part, y)
        else:
            setattr(a, x, y)
    size = att._lib.lard_prefix_attn_workspace_bytes(ctypes.byref(a))
    return att._lib.lard_prefix_attn(ctypes.byref(a), ws, size, None)


@pytest.mark.parametrize("kw", [
    dict(P=-1), dict(S=-1), dict(P=0, S=0), dict(n=0), dict(Hq=5), dict(tau=-1.0), dict(kp_ptr=None), dict(vs_ptr=None),
    dict(kp_row=65), dict(vp_head=-64), dict(ks_batch=4), dict(s_len=20 * STEP + 2), dict(out_ptr=STEP),
    dict(lse=None), dict(P=100000, ws=40 * STEP + 8), dict(P=100000, ws=None), dict(P=100000, ws=6 * STEP),
])
def test_prefix_refuses(att, kw):
    assert prefix_call(att, **kw) == 1


FAR = 1 << 46  # more than any tensor of the largest sizes


def far(call):
    """Addresses of a call so far apart that tensors of any size are disjoint."""
    names = "q k v out dout dq dk dv" if call is cross_call else "q kp vp ks vs out"
    return {f"{x}_ptr": (i + 1) * FAR for i, x in enumerate(names.split())} | dict(
        lse=20 * FAR, ws=30 * FAR, **({"k_len": 22 * FAR} if call is cross_call else {"s_len": 22 * FAR}))


END = 1 << 31


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("kw,over", [
    (dict(B=1, Hq=1, Hkv=1, n=END - 256), dict(n=END - 255)),
    (dict(B=1, Hq=1, Hkv=1, n=1, m=END - 256), dict(m=END - 255)),
    (dict(B=1, Hq=2, Hkv=1, n=END // 2 - 128), dict(n=END // 2 - 127)),
    (dict(B=1 << 20, Hq=1023, Hkv=1023, n=1, m=1), dict(Hq=1024, Hkv=1024)),
])
def test_size_limits_of_cross_attention(att, dtype, kw, over):
    """The header's limits are those of the checks, in both passes."""
    end = 1 if torch.cuda.is_available() else 3
    for fn in ("fwd", "bwd"):
        assert cross_call(att, fn, **far(cross_call), **dict(kw, dtype=dtype)) == end
        assert cross_call(att, fn, **far(cross_call), **dict(kw, dtype=dtype, **over)) == 1


@pytest.mark.parametrize("fn,dtype,rows", [("fwd", 0, 256), ("bwd", 0, 128), ("fwd", 1, 64), ("bwd", 1, 64)])
def test_limit_of_a_launchs_blocks(att, fn, dtype, rows):
    end = 1 if torch.cuda.is_available() else 3
    size = dict(Hq=1, Hkv=1, n=END - 256, dtype=dtype)  # (END - 256) / rows blocks a sequence
    assert cross_call(att, fn, **far(cross_call), B=rows, **size) == end
    assert cross_call(att, fn, **far(cross_call), B=rows + 1, **size) == 1


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("kw,over", [
    (dict(B=1, Hq=1, Hkv=1, n=END - 256, S=0), dict(n=END - 255)),
    (dict(B=1, Hq=1, Hkv=1, n=1, S=1, P=END - 256), dict(P=END - 255)),
    (dict(B=1, Hq=1, Hkv=1, n=1, P=0, S=END - 256), dict(S=END - 255)),
    (dict(B=2, Hq=2, Hkv=1, n=END // 4 - 64, S=0), dict(n=END // 4 - 63)),          # queries of a key head
    (dict(B=1 << 20, Hq=1023, Hkv=1023, n=1, S=0), dict(Hq=1024, Hkv=1024)),
    (dict(B=2, Hq=16, Hkv=16, n=END // 32 - 8), dict(n=END // 32)),                  # rows to join
])
def test_size_limits_of_prefix_attention(att, dtype, kw, over):
    end = 1 if torch.cuda.is_available() else 3
    assert prefix_call(att, **far(prefix_call), **dict(kw, dtype=dtype)) == end
    assert prefix_call(att, **far(prefix_call), **dict(kw, dtype=dtype, **over)) == 1


def test_null_arguments(att):
    assert att._lib.lard_cross_attn_fwd(None, None, 0, None) == 1
    assert att._lib.lard_cross_attn_bwd(None, None, 0, None) == 1
    assert att._lib.lard_prefix_attn(None, None, 0, None) == 1
    assert att._lib.lard_cross_attn_fwd_workspace_bytes(None) == 0
    assert att._lib.lard_prefix_attn_workspace_bytes(None) == 0


def test_binding_refuses(att):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    q, k = z(2, 4, 5, 64), z(2, 2, 7, 64)
    lse, out = z(2, 4, 5, dt=torch.float32), z(2, 4, 5, 64)
    args = lambda **kw: att._cross_args(*[kw.get(x, y) for x, y in (  # noqa: E731
        ("q", q), ("k", k), ("v", k), ("tau", 0.1), ("k_len", None), ("out", out), ("lse", lse))])
    args()
    for bad in (dict(q=q[0]), dict(k=k[0]), dict(v=z(2, 2, 8, 64)), dict(k=z(3, 2, 7, 64)), dict(k=z(2, 2, 7, 32)),
                dict(q=q.half()), dict(k=k.float()), dict(out=out.float()), dict(lse=lse.double()), dict(lse=lse[:1]),
                dict(k_len=z(2)), dict(k_len=z(3, dt=torch.int32)), dict(k_len=z(4, dt=torch.int32)[::2]),
                dict(v=z(2, 2, 64, 7).transpose(2, 3)), dict(lse=z(2, 5, 4, dt=torch.float32).transpose(1, 2))):
        with pytest.raises(ValueError):
            args(**bad)
    with pytest.raises(ValueError):
        att.lard_cross_attn_bwd(q, k, k, 0.1, out, lse, out, q, k, z(2, 2, 7, 64, dt=torch.float32))
    with pytest.raises(ValueError):  # no workspace given where one is needed
        att.lard_cross_attn_bwd(q, k, k, 0.1, out, lse, out, q, k, k)
    with pytest.raises(ValueError):
        att.lard_prefix_attn(q, None, None, None, None, None, 0.1, out, lse)
    with pytest.raises(ValueError):
        att.lard_prefix_attn(q, k[0], None, k, k, None, 0.1, out, lse)
    with pytest.raises(ValueError):
        att.lard_prefix_attn(q, z(3, 9, 64), z(3, 9, 64), k, k, None, 0.1, out, lse)
    with pytest.raises(ValueError):
        att.lard_prefix_attn(q, k, k, k, k, None, 0.1, out, lse)


class _OnGpu1(torch.Tensor):
    """A host tensor that says it is on GPU 1."""

    def get_device(self):
        return 1

    @property
    def device(self):
        return torch.device("cuda", 1)


class _Streams:
    """Stands in for torch's streams, with GPU 0 current: which stream is current on each GPU."""

    def __init__(self):
        self.gpu, self.at = 0, {0: 0xA0, 1: 0xA1}

    def external(self, handle, device=None):
        gpu = self.gpu if device is None else torch.device(device).index
        return types.SimpleNamespace(cuda_stream=handle, device=torch.device("cuda", gpu))

    @contextlib.contextmanager
    def use(self, stream):
        before = self.gpu, dict(self.at)
        self.gpu, self.at[stream.device.index] = stream.device.index, stream.cuda_stream
        yield
        self.gpu, self.at = before


@pytest.mark.parametrize("given", ["raw handle", "stream", "none"])
@pytest.mark.parametrize("call", ["forward", "training step", "prefix"])
def test_work_goes_to_the_given_stream(att, monkeypatch, call, given):
    """The allocating calls enqueue on the stream that they are given, and allocate for it,
    also where the inputs are on a GPU that is not the current one."""
    streams, enqueued, allocated = _Streams(), [], []
    for name in ("lard_cross_attn_fwd", "lard_cross_attn_bwd", "lard_prefix_attn"):
        monkeypatch.setattr(att._lib, name, lambda args, ws, size, stream: enqueued.append(stream) or 0)
    monkeypatch.setattr(att, "_raw_stream", lambda gpu: streams.at[gpu])
    monkeypatch.setattr(torch.cuda, "ExternalStream", streams.external)
    monkeypatch.setattr(torch.cuda, "stream", streams.use)
    monkeypatch.setattr(torch, "empty_strided", lambda size, stride, device, dtype: allocated.append(
        streams.at[device.index]) or torch.zeros(size, dtype=dtype).as_subclass(_OnGpu1))
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16).as_subclass(_OnGpu1)  # noqa: E731
    q, k = z(2, 4, 5, 64), z(2, 2, 7, 64)
    stream = {"raw handle": 0xC0DE, "stream": streams.external(0xC0DE, "cuda:1"), "none": None}[given]
    if call == "prefix":
        att.prefix_attention(q, k[0], k[0], k, k, None, 0.1, stream=stream)
    else:
        att.cross_attention(q, k, k, 0.1, dout=q if call == "training step" else None, stream=stream)
    assert enqueued == [0xA1 if stream is None else 0xC0DE] * (2 if call == "training step" else 1)
    assert allocated and set(allocated) == set(enqueued)
    assert (streams.gpu, streams.at) == (0, {0: 0xA0, 1: 0xA1})


@pytest.mark.parametrize("binding", ["attention", "lard"])
def test_status_is_read_on_the_streams_gpu(att, monkeypatch, binding):
    """The default stream's handle is 0 on every GPU, and the library takes 0 for the current
    GPU's: the binding makes the stream's GPU current."""
    from linear_memory_attention_b200 import lard
    module, name = (att, "lard_attn_device_status") if binding == "attention" else (lard, "lard_device_status")
    gpu, seen = [0], []

    @contextlib.contextmanager
    def device(which):
        before, gpu[0] = gpu[0], torch.device(which).index
        yield
        gpu[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream(0xA0, gpu[0]))
    monkeypatch.setattr(module._lib, name, lambda handle, bits: seen.append((getattr(handle, "value", handle) or 0, gpu[0])) or 0)
    stream = lambda handle, at: types.SimpleNamespace(cuda_stream=handle, device=torch.device("cuda", at))  # noqa: E731
    for given in (stream(0, 1), stream(0xC0DE, 1), stream(0, 0), None, 0xC0DE, 0):
        getattr(module, name)(given)
    assert seen == [(0, 1), (0xC0DE, 1), (0, 0), (0xA0, 0), (0xC0DE, 0), (0, 0)] and gpu == [0]


def test_workspace_grows_with_what_is_split(att):
    """Few rows over many keys are split over blocks, whose partial rows need room; enough
    rows need none."""
    bf = torch.bfloat16
    few, many = torch.empty((1, 8, 1, 128), dtype=bf), torch.empty((8, 32, 1, 128), dtype=bf).expand(8, 32, 4096, 128)
    keys = torch.empty((1, 8, 1, 128), dtype=bf).expand(1, 8, 100000, 128)
    assert att.lard_cross_attn_fwd_workspace_bytes(few, keys) >= 8 * 129 * 4
    assert att.lard_cross_attn_fwd_workspace_bytes(many, keys.expand(8, 8, 100000, 128)) == 0


def test_missing_library_is_an_import_error(tmp_path):
    src = os.path.join(ROOT, "linear_memory_attention_b200")
    pkg = tmp_path / "linear_memory_attention_b200"
    pkg.mkdir()
    for f in ("__init__.py", "lard.py", "attention.py"):
        (pkg / f).write_text(open(os.path.join(src, f)).read())
    os.symlink(os.path.join(src, "liblard.so"), pkg / "liblard.so")
    out = subprocess.run([sys.executable, "-c", "import linear_memory_attention_b200.attention"], cwd=tmp_path,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode != 0 and "ImportError" in out.stderr and "liblard_attn.so is not built" in out.stderr
