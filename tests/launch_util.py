"""What a call launches: the call is captured into a graph that is never run,
and the graph's kernel nodes are read."""
from __future__ import annotations

import ctypes

import torch

_vp, _u32 = ctypes.c_void_p, ctypes.c_uint
THREAD_LOCAL, CLUSTER_DIMENSION = 1, 4


class _KernelNode(ctypes.Structure):
    _fields_ = [("func", _vp), ("grid", _u32 * 3), ("block", _u32 * 3), ("shared", _u32), ("params", _vp), ("extra", _vp), ("kern", _vp),
                ("ctx", _vp)]


def _cuda(name, *args):
    rc = getattr(ctypes.CDLL("libcuda.so.1"), name)(*args)
    assert rc == 0, f"{name}: {rc}"


def _name(node):
    name = ctypes.c_char_p()
    if node.func:
        _cuda("cuFuncGetName", ctypes.byref(name), _vp(node.func))
    else:
        _cuda("cuKernelGetName", ctypes.byref(name), _vp(node.kern))
    return name.value.decode()


def launches(call):
    """(kernel's mangled name, CTAs, CTAs of a cluster) of each kernel that call(stream) launches."""
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    s, graph, n = _vp(stream.cuda_stream), _vp(), ctypes.c_size_t()
    _cuda("cuStreamBeginCapture_v2", s, THREAD_LOCAL)
    try:
        call(stream)
    finally:
        _cuda("cuStreamEndCapture", s, ctypes.byref(graph))
    _cuda("cuGraphGetNodes", graph, None, ctypes.byref(n))
    nodes = (_vp * n.value)()
    _cuda("cuGraphGetNodes", graph, nodes, ctypes.byref(n))
    found = []
    for at in nodes:
        node, value = _KernelNode(), (_u32 * 16)()
        _cuda("cuGraphKernelNodeGetParams_v2", _vp(at), ctypes.byref(node))
        _cuda("cuGraphKernelNodeGetAttribute", _vp(at), CLUSTER_DIMENSION, value)
        found.append((_name(node), node.grid[0] * node.grid[1] * node.grid[2], max(1, value[0])))
    _cuda("cuGraphDestroy", graph)
    return found
