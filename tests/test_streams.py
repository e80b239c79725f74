"""The binding's own work on the host: the buffers that a call allocates belong
to the stream it is queued on, a cache's tensors stay, the tensors of a call
are on one device.  A stand-in for a CUDA tensor notes the stream it was
allocated on, and a stand-in library takes the call."""
import contextlib
import types

import pytest


class _Tensor:
    is_cuda = property(lambda self: self.index >= 0)

    def __init__(self, world, shape, dtype, stream="made by the caller"):
        import torch

        self.world, self.shape, self.dtype, self.stream = world, torch.Size(shape), dtype, stream
        self.used = []
        world.made.append(self)

    device = "cuda:0"
    data_ptr = lambda self: 4096 * (1 + self.world.made.index(self))
    is_contiguous = lambda self: True
    index = 0
    get_device = lambda self: self.index
    numel = lambda self: self.shape.numel()
    element_size = lambda self: self.dtype.itemsize
    nbytes = property(lambda self: self.numel() * self.element_size())
    dim = lambda self: len(self.shape)

    def new_empty(self, shape, dtype=None):
        shape = (shape,) if isinstance(shape, int) else shape
        return _Tensor(self.world, shape, dtype or self.dtype, self.world.current)

    def record_stream(self, stream):
        self.used.append(stream)


@pytest.fixture
def world(monkeypatch):
    import torch

    import ternary_weight_ptq1_gb300 as P

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    w = types.SimpleNamespace(P=P, made=[], calls=[], main=Stream(1), side=Stream(2))
    w.current = w.main

    @contextlib.contextmanager
    def on(stream):
        before, w.current = w.current, stream
        yield
        w.current = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("workspace_bytes"):
                    return 1 << 20
                w.calls.append((name, args))
                return 0
            return call

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=None, device=None: _Tensor(
        w, shape[0] if isinstance(shape[0], tuple) else shape, dtype, w.current))
    monkeypatch.setattr(torch, "empty_like", lambda t: t.new_empty(t.shape))
    monkeypatch.setattr(P, "load", lambda path=None: Library())
    raw = lambda device: w.current.cuda_stream  # noqa: E731
    monkeypatch.setattr(P, "_raw_stream", raw)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", raw, raising=False)
    w.new = lambda shape, dtype: _Tensor(w, shape, dtype)
    return w


def _calls(w):
    import torch

    P, new = w.P, w.new
    f32, bf16, i8, i16, i32, u8 = (torch.float32, torch.bfloat16, torch.int8, torch.int16, torch.int32, torch.uint8)
    x, wq, sc, sg = new((4, 1024), f32), new((256, 208), u8), new((256, 8), i16), new((1024,), i8)
    ids = new((4,), i32)
    cache = types.SimpleNamespace(kv_heads=2, head_dim=64, _int32=i32, _bfloat16=bf16, _ref=64, _on=0, k=new((1, 2, 4, 64), i8))
    q, k, cu = new((4, 4, 64), bf16), new((4, 2, 64), bf16), new((2,), i32)
    block = (new((2048, 208), u8), sc, wq, sc, sg, sg)
    return {
        "matmul_f32_peel": lambda **s: P.matmul_f32_peel(wq, sc, x, **s),
        "unpack": lambda **s: P.unpack(wq, 1024, **s),
        "fwht": lambda **s: P.fwht(x, sg, **s),
        "matmul": lambda **s: P.matmul(wq, sc, x, **s),
        "accumulator": lambda **s: P.matmul_bf16_accumulator(wq, sc, new((4, 1024), bf16), **s),
        "pq2_unpack": lambda **s: P.pq2_unpack(wq, 1024, **s),
        "matmul_pq2": lambda **s: P.matmul_pq2(wq, sc, x, **s),
        "rotate_matmul": lambda **s: P.rotate_matmul(wq, sc, x, sg, **s),
        "ffn": lambda **s: P.ffn(*block, x, **s),
        "ffn_noalloc": lambda **s: P.ffn_noalloc(*block, x, **s),
        "embed": lambda **s: P.embed(x, ids, sg, **s),
        "embed_ptq1": lambda **s: P.embed_ptq1(wq, sc, ids, sg, **s),
        "kv_read": lambda **s: P.kv_read(cache, ids, **s),
        "attn_decode": lambda **s: P.attn_decode(q, cache, new((4, 3), i32), ids, **s),
        "attn_prefill": lambda **s: P.attn_prefill(q, k, k, cu, cu, **s),
    }


NAMES = ("matmul_f32_peel", "unpack", "fwht", "matmul", "accumulator", "pq2_unpack", "matmul_pq2", "rotate_matmul",
         "ffn", "ffn_noalloc", "embed", "embed_ptq1", "kv_read", "attn_decode", "attn_prefill")


@pytest.mark.parametrize("name", NAMES)
def test_buffers_belong_to_the_calls_stream(world, name):
    call = _calls(world)[name]
    n = len(world.made)
    back = call(stream=world.side)
    made = [t for t in world.made[n:] if t.stream != "made by the caller"]
    assert made and all(t.stream is world.side for t in made), [t.shape for t in made if t.stream is not world.side]
    # what the caller gets is used on its current stream too
    for t in back if isinstance(back, tuple) else (back,):
        assert t.used == [world.main]
    (_, args), = world.calls
    assert args[-1] == 2                    # queued on the side stream


@pytest.mark.parametrize("name", NAMES)
def test_without_a_stream_they_belong_to_the_current_one(world, name):
    call = _calls(world)[name]
    n = len(world.made)
    call()
    made = [t for t in world.made[n:] if t.stream != "made by the caller"]
    assert made and all(t.stream is world.main and not t.used for t in made)


# ---- kv_read's results -------------------------------------------------------------

def _cache(w, dtype=None):
    import torch

    dtype = dtype or torch.bfloat16
    k, v = (w.new((3, 2, 4, 64), dtype) for _ in range(2))
    scales = [w.new((3, 2, 4), torch.float32) for _ in range(2)] if dtype == torch.int8 else []
    return w.P.KVCache(k, v, *scales)


@pytest.mark.parametrize("given", ["k", "v"])
def test_the_result_beside_a_given_one_is_of_its_type(world, given):
    import torch

    ids, mine = world.new((4,), torch.int32), world.new((4, 2, 64), torch.float32)
    k, v = world.P.kv_read(_cache(world), ids, **{given: mine})
    assert (k if given == "k" else v) is mine and k.dtype == v.dtype == torch.float32


# ---- the cache object ----------------------------------------------------------------

@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "pages", "page_tokens", "kv_heads", "head_dim"])
def test_a_caches_tensors_are_not_replaced(world, name):
    """The library has their addresses: another tensor would be ignored."""
    import torch

    cache = _cache(world, torch.int8)
    was = getattr(cache, name)
    with pytest.raises(AttributeError, match=name):
        setattr(cache, name, was)
    assert getattr(cache, name) is was


# ---- devices -------------------------------------------------------------------------

def _attention(w):
    """The attention calls by name, and the tensors of each."""
    import torch

    P, new = w.P, w.new
    f32, bf16, i8, i32, u8 = torch.float32, torch.bfloat16, torch.int8, torch.int32, torch.uint8
    cache = _cache(w)
    t = dict(k=new((4, 2, 64), bf16), v=new((4, 2, 64), bf16), slots=new((4,), i32), q=new((4, 4, 64), bf16),
             out=new((4, 4, 64), bf16), lse=new((4, 4), f32), workspace=new((1 << 20,), u8), table=new((4, 3), i32),
             lens=new((4,), i32), cu_q=new((3,), i32), cu_k=new((3,), i32))
    some = lambda *names: {n: t[n] for n in names}  # noqa: E731
    rest = some("out", "lse", "workspace")
    pools = {n: new((3, 2, 4, 64) if n in "kv" else (3, 2, 4), i8 if n in "kv" else f32)
             for n in ("k", "v", "k_scale", "v_scale")}
    return {
        "KVCache": (lambda: P.KVCache(**pools), pools),
        "kv_write": (lambda: P.kv_write(cache, t["k"], t["v"], t["slots"]), some("k", "v", "slots")),
        "kv_read": (lambda: P.kv_read(cache, t["slots"], k=t["k"], v=t["v"]), some("k", "v", "slots")),
        "attn_decode": (lambda: P.attn_decode(t["q"], cache, t["table"], t["lens"], **rest),
                        some("q", "table", "lens", "out", "lse", "workspace")),
        "attn_prefill": (lambda: P.attn_prefill(t["q"], t["k"], t["v"], t["cu_q"], t["cu_k"], **rest),
                         some("q", "k", "v", "cu_q", "cu_k", "out", "lse", "workspace")),
    }


@pytest.mark.parametrize("name", ["KVCache", "kv_write", "kv_read", "attn_decode", "attn_prefill"])
def test_tensors_of_one_call_are_on_one_device(world, name):
    call, tensors = _attention(world)[name]
    call()
    done = len(world.calls)
    for n, t in tensors.items():
        t.index = 1
        with pytest.raises(ValueError, match="device"):
            call()
        t.index = -1                        # the host
        with pytest.raises(TypeError, match="CUDA"):
            call()
        t.index = 0
    assert len(world.calls) == done


def test_an_array_is_no_tensor(world):
    import numpy as np
    import torch

    P, new = world.P, world.new
    q, lens, cache = new((4, 4, 64), torch.bfloat16), new((4,), torch.int32), _cache(world)
    with pytest.raises(TypeError, match="table must be a CUDA tensor"):
        P.attn_decode(q, cache, np.zeros((4, 3), np.int32), lens)
    with pytest.raises(TypeError, match="cu_q must be a CUDA tensor"):
        k = new((4, 2, 64), torch.bfloat16)
        cu = types.SimpleNamespace(numel=lambda: 3, shape=(3,))
        P.attn_prefill(q, k, k, cu, cu)
    assert not world.calls
