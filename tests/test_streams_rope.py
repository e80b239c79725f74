"""The binding's own work on the host for norms with rotation, appending, chunks
and windows: whose stream buffers belong to, that the tensors of a call are on
one device, what is refused (stand-ins as in test_streams)."""
import pytest

from test_streams import _cache, world  # noqa: F401


def _things(w):
    import torch

    P, new = w.P, w.new
    f32, bf16, i8, i32, u8 = torch.float32, torch.bfloat16, torch.int8, torch.int32, torch.uint8
    cache = _cache(w)
    r = dict(inv_freq=new((32,), f32), axis=new((32,), i8), q_gain=new((64,), f32), k_gain=new((64,), f32))
    t = dict(q=new((4, 4, 64), bf16), k=new((4, 2, 64), bf16), v=new((4, 2, 64), bf16), pos=new((2, 4), i32),
             slots=new((4,), i32), table=new((2, 3), i32), lens=new((2,), i32), cu_q=new((3,), i32),
             q_out=new((4, 4, 64), bf16), k_out=new((4, 2, 64), bf16), out=new((4, 4, 64), bf16), lse=new((4, 4), f32),
             workspace=new((1 << 20,), u8), table4=new((4, 3), i32), lens4=new((4,), i32))
    return P, cache, r, t


def _calls(w):
    P, cache, r, t = _things(w)
    rope = P.Rope(**r)
    return {
        "qk_rope": lambda **s: P.qk_rope(rope, t["q"], t["k"], t["pos"], **s),
        "kv_append": lambda **s: P.kv_append(cache, rope, t["k"], t["v"], t["slots"], t["pos"], q=t["q"], **s),
        "attn_chunk": lambda **s: P.attn_chunk(t["q"], cache, t["table"], t["lens"], t["cu_q"], **s),
        "attn_decode": lambda **s: P.attn_decode(t["q"], cache, t["table4"], t["lens4"], window=7, sinks=2, **s),
    }


NAMES = ("qk_rope", "kv_append", "attn_chunk", "attn_decode")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("side", [True, False])
def test_buffers_belong_to_the_calls_stream(world, name, side):  # noqa: F811
    call = _calls(world)[name]
    n = len(world.made)
    back = call(stream=world.side) if side else call()
    made = [t for t in world.made[n:] if t.stream != "made by the caller"]
    assert made and all(t.stream is (world.side if side else world.main) for t in made)
    for t in back if isinstance(back, tuple) else (back,):
        assert t.used == ([world.main] if side else [])
    (_, args), = world.calls
    assert args[-1] == (2 if side else 1)


def test_a_window_is_a_call_of_its_own(world):  # noqa: F811
    P, cache, _, t = _things(world)
    P.attn_decode(t["q"], cache, t["table4"], t["lens4"], sinks=3)
    P.attn_decode(t["q"], cache, t["table4"], t["lens4"], window=9, sinks=3)
    assert [n for n, _ in world.calls] == ["ptq_attn_decode", "ptq_attn_decode_window"]
    assert world.calls[1][1][11:13] == (9, 3)


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_one_call_are_on_one_device(world, name):  # noqa: F811
    P, cache, r, t = _things(world)
    rope = P.Rope(**r)
    rest = {n: t[n] for n in ("out", "lse", "workspace")}
    call, names = {
        "qk_rope": (lambda: P.qk_rope(rope, t["q"], t["k"], t["pos"], q_out=t["q_out"], k_out=t["k_out"]),
                    ("k", "pos", "q_out", "k_out")),
        "kv_append": (lambda: P.kv_append(cache, rope, t["k"], t["v"], t["slots"], t["pos"], q=t["q"], q_out=t["q_out"]),
                      ("q", "k", "v", "slots", "pos", "q_out")),
        "attn_chunk": (lambda: P.attn_chunk(t["q"], cache, t["table"], t["lens"], t["cu_q"], **rest),
                       ("q", "table", "lens", "cu_q", "out", "lse", "workspace")),
        "attn_decode": (lambda: P.attn_decode(t["q"], cache, t["table4"], t["lens4"], window=3, **rest),
                        ("q", "table4", "lens4", "out", "lse", "workspace")),
    }[name]
    call()
    done = len(world.calls)
    for n in names:
        t[n].index = 1
        with pytest.raises(ValueError, match="device"):
            call()
        t[n].index = -1                        # the host
        with pytest.raises(TypeError, match="CUDA"):
            call()
        t[n].index = 0
    assert len(world.calls) == done


def test_a_rope_on_another_device_and_one_that_is_changed(world):  # noqa: F811
    P, cache, r, t = _things(world)
    rope = P.Rope(**r)
    with pytest.raises(AttributeError, match="not replaced"):
        rope.inv_freq = r["inv_freq"]
    for x in r.values():
        x.index = 1
    other = P.Rope(**r)
    with pytest.raises(ValueError, match="device"):
        P.qk_rope(other, t["q"], t["k"], t["pos"])
    r["axis"].index = 0
    with pytest.raises(ValueError, match="device"):
        P.Rope(**r)
    assert not world.calls


def test_shapes_that_do_not_fit(world):  # noqa: F811
    import torch

    P, cache, r, t = _things(world)
    rope, new = P.Rope(**r), world.new
    bf16, i32 = torch.bfloat16, torch.int32
    with pytest.raises(ValueError, match="k must be"):
        P.qk_rope(rope, t["q"], new((5, 2, 64), bf16), t["pos"])
    with pytest.raises(ValueError, match="pos must be"):
        P.qk_rope(rope, t["q"], t["k"], new((2, 5), i32))
    with pytest.raises(ValueError, match="q_gain must be"):
        P.qk_rope(rope, new((4, 4, 128), bf16), new((4, 2, 128), bf16), t["pos"])
    with pytest.raises(ValueError, match="q_out"):
        P.qk_rope(rope, t["q"], t["k"], t["pos"], q_out=new((4, 3, 64), bf16))
    with pytest.raises(TypeError, match="k must be"):
        P.qk_rope(rope, t["q"], new((4, 2, 64), torch.float32), t["pos"])
    with pytest.raises(ValueError, match="q must be"):
        P.kv_append(cache, rope, t["k"], t["v"], t["slots"], t["pos"], q=new((5, 4, 64), bf16))
    with pytest.raises(ValueError, match="without q"):
        P.kv_append(cache, rope, t["k"], t["v"], t["slots"], t["pos"], q_out=t["q_out"])
    with pytest.raises(ValueError, match="k must be"):
        P.kv_append(cache, rope, new((4, 3, 64), bf16), t["v"], t["slots"], t["pos"])
    with pytest.raises(ValueError, match="cu_q must have"):
        P.attn_chunk(t["q"], cache, t["table"], t["lens"], new((4,), i32))
    with pytest.raises(ValueError, match="head_dim"):
        P.attn_chunk(new((4, 4, 128), bf16), cache, t["table"], t["lens"], t["cu_q"])
    assert not world.calls


def test_a_rope_in_two_threads(world):  # noqa: F811
    """Each thread has a struct of its own: positions of one call are not another's."""
    import threading

    P, _, r, t = _things(world)
    rope = P.Rope(**r)
    import torch

    other = world.new((4,), torch.int32)
    got, both = {}, threading.Barrier(2)

    def call(name, pos):
        at = rope._at(pos, 4, 64, 0)
        both.wait()
        s = P._RopeStruct.from_address(at)
        got[name] = at, s.pos, s.axes
        both.wait()

    threads = [threading.Thread(target=call, args=a) for a in (("a", t["pos"]), ("b", other))]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert got["a"][0] != got["b"][0]
    assert got["a"][1:] == (t["pos"].data_ptr(), 2) and got["b"][1:] == (other.data_ptr(), 1)
