"""What the binding makes for a call that is given a stream (copies of views,
outputs, workspaces, plans) is made on that stream, and what it leaves in use
there is not handed out again too early.  No GPU: the library and torch's device
side are stand-ins that write down under which stream each thing was asked for."""
import contextlib
import types

import pytest
import torch

from attention_forward_online_gb300 import osattn

MAIN, SIDE = 11, 22


class World:
    def __init__(self):
        self.current, self.log, self.lent = MAIN, [], []


class Tensor:
    """A CUDA tensor's outside; `contiguous` makes a copy if it is a view."""

    def __init__(self, world, shape, dtype, name, view=False, strides=None):
        self.world, self.shape, self.dtype, self.name, self.view = world, torch.Size(shape), dtype, name, view
        self.is_cuda, self.device = True, torch.device("cuda", 0)
        size = 1
        st = []
        for n in reversed(shape):
            st.insert(0, size)
            size *= n
        self.size, self.st = size, tuple(strides or st)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self.st if i is None else self.st[i]

    def numel(self):
        return self.size

    def element_size(self):
        return 1

    def get_device(self):
        return 0

    def is_contiguous(self):
        return not self.view

    def contiguous(self):
        if not self.view:
            return self
        self.world.log.append((self.name + " copy", self.world.current))
        return Tensor(self.world, self.shape, self.dtype, self.name)

    def data_ptr(self):
        return 0x10000

    def new_empty(self, shape, dtype=None):
        shape = (shape,) if isinstance(shape, int) else shape
        return self.world.empty(shape, dtype or self.dtype)

    def record_stream(self, stream):
        self.world.lent.append((self.name, stream.cuda_stream))


def stream(handle):
    return types.SimpleNamespace(cuda_stream=handle, device=torch.device("cuda", 0), device_index=0)


@pytest.fixture
def world(monkeypatch):
    w = World()

    def empty(shape, dtype=None, device=None):
        shape = (shape,) if isinstance(shape, int) else tuple(shape)
        w.log.append(("allocation", w.current))
        return Tensor(w, shape, dtype, "made")

    @contextlib.contextmanager
    def under(s):
        before, w.current = w.current, s.cuda_stream
        yield
        w.current = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                handle = args[-1]
                w.log.append((name, getattr(handle, "value", handle)))
                return 0
            return call

    w.empty = empty
    monkeypatch.setattr(osattn, "_lib", Library())
    monkeypatch.setattr(osattn, "lib", lambda: osattn._lib)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape, t.dtype))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream(w.current))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: w.current, raising=False)
    for name in ("bwd_workspace_bytes", "splitkv_workspace_bytes"):
        monkeypatch.setattr(osattn, name, lambda *a: 64)
    return w


def qkv(w, Hkv=2, N=8):
    t = torch.bfloat16
    return [Tensor(w, (1, h, N, 64), t, n) for h, n in ((4, "q"), (Hkv, "k"), (Hkv, "v"))]


def view(w, shape, dtype, name):
    return Tensor(w, shape, dtype, name, view=True)


def plan_of(w, s=None):
    return osattn.mask_plan(1, 8, 8, causal=True, device="cuda:0", stream=s)


def calls(w, s):
    t = torch.bfloat16
    q, k, v = qkv(w)
    i32 = torch.int32
    score = dict(rel_table=view(w, (5, 4), t, "table"), rel_map=view(w, (3,), i32, "map"))
    lse = Tensor(w, (1, 4, 8), torch.float32, "lse")
    pages = [Tensor(w, (6, 2, 16, 64), t, n) for n in ("kp", "vp")]
    f = [Tensor(w, (1, 4, 8, 64), t, n) for n in ("q", "k", "v")]
    kl = view(w, (1,), i32, "key_len")
    return {
        "mask_plan": lambda: osattn.mask_plan(1, 8, 8, key_len=kl, doc_ids=view(w, (1, 8), i32, "docs"), stream=s),
        "fwd_mod": lambda: osattn.fwd_mod(q, k, v, stream=s, **score),
        "slopes": lambda: osattn.fwd_mod(q, k, v, slopes=view(w, (4,), torch.float32, "slopes"), stream=s),
        "bwd_mod": lambda: osattn.bwd_mod(q, k, v, q, lse, q, stream=s, **score),
        "tree_attn": lambda: osattn.tree_attn(q, *pages, view(w, (1, 4), i32, "pages"), view(w, (1,), i32, "ctx"),
                                              view(w, (1, 8), torch.int64, "mask"), stream=s),
        "fwd": lambda: osattn.fwd(*f, key_len=kl, stream=s),
        "fwd_splitkv": lambda: osattn.fwd_splitkv(*f, 2, key_len=kl, stream=s),
        "bwd": lambda: osattn.bwd(*f, f[0], lse, f[0], key_len=kl, stream=s),
        "softmax_rows": lambda: osattn.softmax_rows(Tensor(w, (4, 8), t, "x"), stream=s),
    }


NAMES = ["mask_plan", "fwd_mod", "slopes", "bwd_mod", "tree_attn", "fwd", "fwd_splitkv", "bwd", "softmax_rows"]


@pytest.mark.parametrize("name", NAMES)
def test_everything_is_made_on_the_stream_of_the_call(world, name):
    results = calls(world, stream(SIDE))[name]()
    launches = [x for x in world.log if x[0].startswith("osattn_")]
    assert len(launches) == 1 and len(world.log) > 1
    assert {s for _, s in world.log} == {SIDE}, world.log
    assert world.current == MAIN
    # results that the caller's stream goes on to use are not reused under it
    made = 1 if name == "mask_plan" else len([r for r in results if r is not None])
    assert world.lent.count(("made", MAIN)) >= made


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_needs_nothing_of_it(world, name):
    for s in (None, stream(MAIN)):
        world.log.clear()
        calls(world, s)[name]()
        assert {x for _, x in world.log} == {MAIN} and not world.lent
