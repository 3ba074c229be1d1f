"""Child process of tests/test_gpu_per_head_timeout.py.

Usage: python per_head_timeout_child.py <failure-detection library>

Runs the window attention of two requests with 80 new tokens each, whole and
in two ranges through a workspace, with the failure-detection build of the
library (the warp that issues the output products stops at a fixed tile, so
that the other roles' bounded waits run out), then with the normal one, and
reports in JSON on stdout: per call the status words, whether the stalled call
left its outputs as they were, and whether the normal call after it gives the
bits of the normal call before it.
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
    B, new, H, KH, D, block, context = 2, 80, 8, 2, 128, 16, 400
    width = (context + new) // block
    cache = torch.from_numpy(rng.integers(0, 256, (B * width, 2, block, KH, D // 2 + D // 16), dtype=np.uint8))
    flat = cache.view(B * width, 2, -1)
    flat[:, :, block * KH * D // 2:] = 0x38                                  # every scale 1
    i32 = dict(dtype=torch.int32, device=dev)
    call = dict(q=torch.from_numpy(rng.standard_normal((B * new, H, D), dtype=np.float32)).to(dev, torch.bfloat16),
                query_start=torch.tensor([0, new, 2 * new], **i32),
                seq_lens=torch.tensor([context + new] * B, **i32),
                block_table=torch.arange(B * width, **i32).view(B, width), kv_cache=cache.to(dev),
                k_scale=torch.ones(1, device=dev), v_scale=torch.ones(1, device=dev), softmax_scale=D ** -0.5,
                max_query_len=new, max_seq_len=context + new)
    stall = ctypes.CDLL(sys.argv[1])
    native = kvq._load_native()
    normal = kvq.load_library()

    def bind(lib):
        native.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in kvq._NATIVE_ENTRIES})

    def run(splits):
        out = torch.full((B * new, H, D), SENTINEL, dtype=torch.bfloat16, device=dev)
        lse = torch.full((B * new, H), SENTINEL, dtype=torch.float32, device=dev)
        status = torch.zeros(1, **i32)
        kvq.kvq_window_attention_nvfp4_per_head(**call, num_splits=splits, out=out, lse=lse, status=status)
        torch.cuda.synchronize(dev)
        return out, lse, int(status.item())

    report = []
    for splits in (1, 2):
        before = run(splits)
        bind(stall)
        out, lse, status = run(splits)
        bind(normal)
        after = run(splits)
        report.append({"splits": splits, "status": status, "normal_status": before[2] | after[2],
                       "untouched": bool(torch.all(out == SENTINEL).item() and torch.all(lse == SENTINEL).item()),
                       "same": bool(torch.equal(before[0].view(torch.int16), after[0].view(torch.int16))
                                    and torch.equal(before[1], after[1])),
                       "finite": bool(torch.isfinite(after[0].float()).all().item())})
    print(json.dumps(report))


if __name__ == "__main__":
    main()
