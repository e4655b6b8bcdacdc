"""The prompt and draft calls refuse tensors that are not all on the current device (its
scratch and its SMs are what a call uses). Shapes alone, no device memory."""
import pytest
import torch
from torch._subclasses import FakeTensorMode

import bit_weight_only_w4a16_gb300 as w4


def calls(where):
    """The calls with every tensor in its place; where(name) is a tensor's device."""
    def make(name, *s, dtype=torch.bfloat16):
        return torch.empty(s, dtype=dtype, device=where(name))

    def i32(name, *s):
        return make(name, *s, dtype=torch.int32)

    def f32(name, *s):
        return make(name, *s, dtype=torch.float32)

    return {
        "prompt": lambda: w4.w4_attn_prompt(make("q", 4, 8, 64), make("k", 4, 1, 64), make("v", 4, 1, 64), i32("cu_q", 2),
                                            i32("cu_k", 2), out=make("out", 4, 8, 64)),
        "tree": lambda: w4.w4_attn_tree(make("q", 1, 4, 8, 64), make("k", 1, 9, 1, 64), make("v", 1, 9, 1, 64),
                                        make("k_tree", 1, 4, 1, 64), make("v_tree", 1, 4, 1, 64), i32("parents", 1, 4),
                                        i32("pos", 1), kpos=i32("kpos", 1, 9), out=make("out", 1, 4, 8, 64)),
        "logprobs": lambda: w4.w4_logprobs(f32("logits", 3, 50), i32("targets", 3), 2, status=i32("status", 1),
                                           out=(f32("logprob", 3), f32("entropy", 3), f32("top_logprob", 3, 2),
                                                i32("top_id", 3, 2))),
        "commit": lambda: w4.w4_kv_commit(make("k_cache", 1, 1, 9, 64), make("v_cache", 1, 1, 9, 64),
                                          make("k_tree", 1, 1, 4, 64), make("v_tree", 1, 1, 4, 64), i32("path", 1, 4),
                                          i32("count", 1), i32("pos", 1), kpos=i32("kpos", 1, 9), status=i32("status", 1)),
    }


TENSORS = {
    "prompt": ["q", "k", "v", "cu_q", "cu_k", "out"],
    "tree": ["q", "k", "v", "k_tree", "v_tree", "parents", "pos", "kpos", "out"],
    "logprobs": ["logits", "targets", "status", "logprob", "entropy", "top_logprob", "top_id"],
    "commit": ["k_cache", "v_cache", "k_tree", "v_tree", "path", "count", "pos", "kpos", "status"],
}


@pytest.mark.parametrize("call,odd", [(c, t) for c, ts in TENSORS.items() for t in ts])
@pytest.mark.parametrize("other", ["cuda:1", "cpu"])
def test_one_tensor_elsewhere(monkeypatch, call, odd, other):
    monkeypatch.setattr(w4, "_current_device", lambda: 0)
    with FakeTensorMode():
        with pytest.raises(ValueError, match="device|CUDA"):
            calls(lambda name: other if name == odd else "cuda:0")[call]()


@pytest.mark.parametrize("call", list(TENSORS))
def test_all_on_another_device_than_the_current_one(monkeypatch, call):
    monkeypatch.setattr(w4, "_current_device", lambda: 0)
    with FakeTensorMode():
        with pytest.raises(ValueError, match="current device is 0"):
            calls(lambda name: "cuda:1")[call]()
