"""Child process of tests/test_gpu_fp8_timeout.py.

Usage: python fp8_timeout_child.py <failure-detection library>

Runs the attention over the e4m3 cache (two requests with 80 new tokens each:
whole, in two ranges through a workspace, over gathered entries) and over two
prompts with the failure-detection build of the library, then with the normal
one, and reports in JSON on stdout: per call the status words, whether the
rows that see more than the tiles before the stall are as they were, whether
every other row is untouched or right, and whether the normal call after it
gives the bits of the normal call before it.
"""
import ctypes
import json
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import fp8_quantized_paged_concat_gb300 as kvq  # noqa: E402

SENTINEL = -7.0


def main():
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    rng = np.random.default_rng(5)
    i32 = dict(dtype=torch.int32, device=dev)
    stall = ctypes.CDLL(sys.argv[1])
    native = kvq._load_native()
    normal = kvq.load_library()

    def bind(lib):
        native.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in kvq._NATIVE_ENTRIES})

    def bf16(*shape):
        return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(dev, torch.bfloat16)

    B, new, H, KH, D, block, context = 2, 80, 8, 2, 128, 16, 400
    width = (context + new) // block
    codes = rng.integers(0, 256, (B * width, 2, block, KH, D), dtype=np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38                             # no NaN
    cached = dict(q=bf16(B * new, H, D), query_start=torch.tensor([0, new, 2 * new], **i32),
                  seq_lens=torch.tensor([context + new] * B, **i32),
                  block_table=torch.arange(B * width, **i32).view(B, width), kv_cache=torch.from_numpy(codes).to(dev),
                  kv_scales=torch.full((B * width, 2, KH), kvq.FP8_SCALE_BIAS - 8, dtype=torch.uint8, device=dev),
                  softmax_scale=D ** -0.5, max_query_len=new, max_seq_len=context + new)
    held = torch.empty(kvq.kvq_fp8_attention_workspace_bytes(B * new, H, KH, D, B, new, context + new), dtype=torch.uint8,
                       device=dev)
    calls = [("whole", kvq.kvq_window_attention_fp8_per_head, dict(cached, num_splits=1), 0),
             ("ranges", kvq.kvq_window_attention_fp8_per_head, dict(cached, num_splits=2), 0),
             ("gathered", kvq.kvq_window_attention_fp8_per_head, dict(cached, num_splits=1, workspace=held), 0)]
    lens = [300, 500]
    for dim in (64, 128, 256):
        qkv = bf16(sum(lens), H + 2 * KH, dim)
        # a block of query rows is 64 tokens or fewer, a tile 64 keys: from token 192 on rows see a third tile
        calls.append((f"prompt {dim}", kvq.kvq_prompt_attention,
                      dict(q=qkv[:, :H], k=qkv[:, H:H + KH], v=qkv[:, H + KH:],
                           seq_start=torch.tensor([0, lens[0], sum(lens)], **i32), softmax_scale=dim ** -0.5,
                           max_seq_len=max(lens)), 192))

    def run(f, call):
        out = torch.full(call["q"].shape, SENTINEL, dtype=torch.bfloat16, device=dev)
        lse = torch.full(call["q"].shape[:2], SENTINEL, dtype=torch.float32, device=dev)
        status = torch.zeros(1, **i32)
        f(**call, out=out, lse=lse, status=status)
        torch.cuda.synchronize(dev)
        return out.float(), lse, int(status.item())

    report = []
    for name, f, call, past in calls:
        before = run(f, call)
        bind(stall)
        out, lse, status = run(f, call)
        bind(normal)
        after = run(f, call)
        kept = (out == SENTINEL).all(2) & (lse == SENTINEL)
        right = (out == before[0]).all(2) & (lse == before[1])
        late = torch.ones(out.shape[0], dtype=torch.bool, device=dev)
        if past:
            late = torch.cat([torch.arange(n, device=dev) >= past for n in lens])
        report.append({"call": name, "status": status, "normal_status": before[2] | after[2],
                       "untouched": bool(kept[late].all().item()), "others": bool((kept | right).all().item()),
                       "same": bool(torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])),
                       "finite": bool(torch.isfinite(after[0]).all().item())})
    print(json.dumps(report))


if __name__ == "__main__":
    main()
