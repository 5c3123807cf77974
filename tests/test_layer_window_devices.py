"""The windowed layer refuses a cache on another GPU than its input, before
anything is enqueued (stand-ins for tensors: no GPU needed)."""
import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from blockwise_attn_ffn_b200 import layer


class Stub:
    """What the front end looks at of a contiguous tensor on a GPU."""

    def __init__(self, index, dtype, *shape):
        self.index, self.dtype, self.shape = index, dtype, torch.Size(shape)
        self.device, self.is_cuda = torch.device("cuda", index), True

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = [1] * len(self.shape)
        for k in range(len(s) - 1, 0, -1):
            s[k - 1] = s[k] * self.shape[k]
        return tuple(s) if i is None else s[i]

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 32  # (never followed: the call itself is replaced)

    def numel(self):
        return self.shape.numel()


def test_a_cache_on_another_gpu_is_refused(monkeypatch):
    called = []
    monkeypatch.setattr(layer, "run", lambda *a: called.append(a) or bpt.BPT_OK)
    monkeypatch.setattr(layer, "current_stream", lambda index: 0)
    B, N, d, h, d_ff = 2, 32, 128, 2, 256
    t = lambda dt, *shape, at=0: Stub(at, dt, *shape)
    bf, f32, i32, f16 = torch.bfloat16, torch.float32, torch.int32, torch.float16
    p = dict(ln1=t(bf, 2, d), W_Q=t(bf, d, d), W_K=t(bf, d, d), W_V=t(bf, d, d), W_O=t(bf, d, d),
             ln2=t(bf, 2, d), W_1=t(bf, d, d_ff), b_1=t(bf, d_ff), W_2=t(bf, d_ff, d), b_2=t(bf, d))
    ws = t(torch.uint8, 1 << 20)

    def go(at):
        cache = (t(f16, 8, h, 16, 64, at=at), t(f16, 8, h, 16, 64, at=at), t(i32, B, 4, at=at),
                 t(i32, B, at=at))
        return bpt.layer_forward_window(t(bf, B, N, d), p, h, 16, out=t(f32, B, N, d), cache=cache,
                                        new_lens=t(i32, B), workspace=ws)

    with pytest.raises(ValueError, match="cuda:0"):
        go(1)
    assert not called
    go(0)
    assert len(called) == 1
