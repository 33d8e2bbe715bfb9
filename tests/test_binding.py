"""The Python binding of the cache and attention calls by itself: which
scratch a call gets, what tensors it takes. On the CPU, with tensors that say
they are on a GPU and a library that only notes its calls."""
import threading
import time

import pytest
import torch

from speculative_decoding_verification_27_gb300 import api, build


class OnGpu(torch.Tensor):
    """A tensor that claims to lie on a GPU."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return getattr(self, "gpu_index", 0)


def gpu(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


class Noted:
    """The library's calls as (name, arguments)."""

    def __init__(self, real):
        self.real, self.calls, self.during = real, [], lambda name, args: None

    def __getattr__(self, name):
        if name.endswith("_size"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            self.during(name, args)
            return 0
        return call

    def blocks(self):
        """The workspaces of the calls so far."""
        at = {"sv_cache_reserve": 6, "sv_window_attention": 14}
        return [args[at[name]].value for name, args in self.calls]


@pytest.fixture
def rig(monkeypatch):
    """(library, cache, page table, lengths, q) with two sequences."""
    build.build_library()
    lib = Noted(api.load())
    monkeypatch.setattr(api, "_new", lambda make, shape, dtype, like, stream: make(shape, dtype=dtype).as_subclass(OnGpu))
    monkeypatch.setattr(api, "_raw_stream", lambda device: 7 + device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    k = gpu(1, 4, 2, 1, 64, dtype=torch.bfloat16)
    cache = api.KVCache(k, k.clone(), gpu(4), gpu(1))
    monkeypatch.setattr(api, "_lib", lib)
    return lib, cache, gpu(2, 3), gpu(2), gpu(2, 1, 64, dtype=torch.bfloat16)


def test_threads_on_one_stream_take_turns(rig):
    """A call of two launches hands its results over in the stream's scratch: no other thread's may come between them."""
    lib, cache, table, ctx, q = rig
    busy, clashes = set(), []

    def during(name, args):
        ws = lib.blocks()[-1]
        clashes.append(ws in busy)
        busy.add(ws)
        time.sleep(0.02)
        busy.discard(ws)

    lib.during = during
    calls = [lambda: api.sv_window_attention(q, cache, 0, table, ctx), lambda: api.sv_cache_reserve(cache, table, ctx)]
    threads = [threading.Thread(target=lambda i=i: [calls[i % 2]() for _ in range(4)]) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(clashes) == 16 and not any(clashes)


def test_capture_is_asked_of_the_caches_device(rig, monkeypatch):
    """The current stream of another device may be capturing, or not be, when the cache's is (not)."""
    lib, cache, table, ctx, q = rig
    current = [1]

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.was, current[0] = current[0], self.device

        def __exit__(self, *e):
            current[0] = self.was

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    blocks = []
    for capturing in (None, 0, 1):  # the device whose current stream captures
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[0] == capturing)
        api.sv_window_attention(q, cache, 0, table, ctx)
        blocks.append(lib.blocks()[-1])
        kept = [s.block.data_ptr() for s in cache._scratches.values()]
        assert kept == blocks[:1]
    assert current == [1]
    assert blocks[2] == blocks[0] != blocks[1]


def test_scratch_is_as_large_as_the_calls_need(rig):
    """A stream that only reserves pages holds a few bytes a sequence; the attention's partial results come with its first call."""
    lib, cache, table, ctx, q = rig
    api.sv_cache_reserve(cache, table, ctx)
    scratch, = cache._scratches.values()
    assert scratch.block.numel() == lib.real.sv_cache_reserve_workspace_size(2)
    api.sv_window_attention(q, cache, 0, table, ctx)
    size = lib.real.sv_window_attention_workspace_size(cache._ref, 1, 2)
    assert scratch.block.numel() == size > 1 << 20
    api.sv_cache_reserve(cache, table, ctx)
    assert scratch.block.numel() == size


def test_tensors_of_another_device_are_refused(rig):
    """Every tensor of a call lies on the cache's (or the logits') device: the kernel reads its address there."""
    lib, cache, table, ctx, q = rig
    i1, i2, i3, i4 = (gpu(n) for n in (1, 2, 3, 4))
    f2, out, ws = gpu(2, dtype=torch.float32), gpu(2, 1, 64, dtype=torch.bfloat16), gpu(1 << 26, dtype=torch.uint8)
    new, z, status = gpu(1, 2, 1, 64, dtype=torch.bfloat16), gpu(2, 8, dtype=torch.float32), gpu(1)
    top_i, top_f = gpu(2, 2), gpu(2, 2, dtype=torch.float32)
    seqs = dict(page_table=table, ctx_len=ctx, status=status)
    win = dict(cu_draft=i3, cu_cand=i3.clone())
    calls = [(api.sv_cache_fork, dict(cache=cache, src=i1, dst=i1.clone(), **seqs)),
             (api.sv_cache_free, dict(cache=cache, which=i1, **seqs)),
             (api.sv_cache_reserve, dict(cache=cache, granted=i2, workspace=ws, **seqs, **win)),
             (api.sv_cache_append, dict(cache=cache, layer=0, k_new=new, v_new=new.clone(), **seqs, **win)),
             (api.sv_cache_commit, dict(cache=cache, out_len=i2, best=i2.clone(), **seqs, **win)),
             (api.sv_window_attention, dict(cache=cache, q=q, layer=0, out=out, out_lse=f2.view(2, 1), workspace=ws, **seqs, **win)),
             (api.sv_token_logprobs, dict(logits=z, tokens=i2, cu_draft=i3, out_len=i2.clone(), n_top=2, out_logprob=f2, out_rank=i2,
                                          out_entropy=f2.clone(), out_top_ids=top_i, out_top_logprobs=top_f, status=status))]
    checked = 0
    for call, args in calls:
        call(**args)
        n = len(lib.calls)
        for name, t in args.items():
            if isinstance(t, torch.Tensor):
                elsewhere = t.clone()
                elsewhere.gpu_index = 1
                with pytest.raises(ValueError):
                    call(**dict(args, **{name: elsewhere}))
                checked += 1
        assert len(lib.calls) == n
    assert checked == 49
    for page_ref, free_bits in ((0, 1), (1, 0)):
        counts = [gpu(4), gpu(1)]
        counts[0].gpu_index, counts[1].gpu_index = page_ref, free_bits
        with pytest.raises(ValueError):
            api.KVCache(cache.k, cache.v, *counts)
