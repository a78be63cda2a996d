"""What a call enqueues: its kernels' names and shapes, from a capture that is never run."""
import ctypes

import torch


class _Params(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _ok(status):
    assert status == 0, f"CUDA status {status}"


def kernels(call, stream):
    """[(name, blocks, threads a block)] of the kernels that call() enqueues on `stream`, sorted by name."""
    cu = ctypes.CDLL("libcuda.so.1")
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    _ok(cu.cuStreamBeginCapture_v2(handle, 2))  # relaxed: the call may allocate
    try:
        with torch.cuda.stream(stream):
            kept = call()
    finally:
        _ok(cu.cuStreamEndCapture(handle, ctypes.byref(graph)))
    count = ctypes.c_size_t()
    _ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(count)))
    nodes = (ctypes.c_void_p * count.value)()
    _ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(count)))
    out = []
    for node in nodes:
        kind = ctypes.c_int()
        _ok(cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)))
        if kind.value != 0:  # not a kernel
            continue
        p, name = _Params(), ctypes.c_char_p()
        _ok(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)))
        if p.func:
            _ok(cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)))
        else:
            _ok(cu.cuKernelGetName(ctypes.byref(name), ctypes.c_void_p(p.kern)))
        out.append((name.value.decode(), p.grid[0] * p.grid[1] * p.grid[2], p.block[0] * p.block[1] * p.block[2]))
    _ok(cu.cuGraphDestroy(graph))
    del kept
    return sorted(out)
