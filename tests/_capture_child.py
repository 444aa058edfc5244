"""The first calls of a process, made while a graph is being captured (run by test_gpu_kv_chunk.py)."""
import sys

import torch

from long_context_decode_bit_b200 import fathom


def main(new: int) -> int:
    dev = "cuda"
    cache = fathom.KVCache.empty(40, 2, 128, 64, dtype=torch.int8)
    table = torch.arange(40, dtype=torch.int32, device=dev)[None]
    cu, length = torch.tensor([0, new], dtype=torch.int32, device=dev), torch.tensor([2000], dtype=torch.int32, device=dev)
    k, v, q = (torch.randn(new, n, 128, device=dev).bfloat16() for n in (2, 2, 8))
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        fathom.kv_write(cache, k, v, table, cu, length)
        out = fathom.paged_attention(cache, q, table, cu, length, new, 2000)
    graph.replay()
    torch.cuda.synchronize()
    want = fathom.paged_attention(cache, q, table, cu, length, new, 2000)
    assert torch.equal(out, want) and bool(out.any()), "replay differs"
    print("same")
    return 0


if __name__ == "__main__":
    sys.exit(main(int(sys.argv[1])))
