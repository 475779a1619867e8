"""The kernels that a call launches, with grid and cluster sizes: the call is
captured in a graph (and not run) and the graph's nodes are read."""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

_CLUSTER_DIMENSION = 4  # CU_LAUNCH_ATTRIBUTE_CLUSTER_DIMENSION


class Launch(NamedTuple):
    name: str      # mangled
    grid: int      # blocks
    cluster: int   # blocks of a cluster


class _KernelNodeParams(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS (v2)
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _ok(status: int, what: str) -> None:
    if status:
        raise RuntimeError(f"{what}: error {status}")


def launches(call) -> list[Launch]:
    """Those of call(), in no order.  call() allocates nothing but tensors."""
    cu = ctypes.CDLL("libcuda.so.1")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    handle = ctypes.c_void_p(graph.raw_cuda_graph())
    n = ctypes.c_size_t(0)
    _ok(cu.cuGraphGetNodes(handle, None, ctypes.byref(n)), "cuGraphGetNodes")
    nodes = (ctypes.c_void_p * n.value)()
    _ok(cu.cuGraphGetNodes(handle, nodes, ctypes.byref(n)), "cuGraphGetNodes")
    out = []
    for node in nodes:
        node, kind = ctypes.c_void_p(node), ctypes.c_int(0)
        _ok(cu.cuGraphNodeGetType(node, ctypes.byref(kind)), "cuGraphNodeGetType")
        if kind.value != 0:  # not a kernel
            continue
        p, name, value = _KernelNodeParams(), ctypes.c_char_p(), (ctypes.c_uint * 16)()
        _ok(cu.cuGraphKernelNodeGetParams_v2(node, ctypes.byref(p)), "cuGraphKernelNodeGetParams")
        if p.func:
            _ok(cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)), "cuFuncGetName")
        else:
            _ok(cu.cuKernelGetName(ctypes.byref(name), ctypes.c_void_p(p.kern)), "cuKernelGetName")
        _ok(cu.cuGraphKernelNodeGetAttribute(node, _CLUSTER_DIMENSION, ctypes.byref(value)),
            "cuGraphKernelNodeGetAttribute")
        out.append(Launch(name.value.decode(), p.grid[0] * p.grid[1] * p.grid[2], max(1, value[0])))
    return out


def the(found: list[Launch], part: str) -> Launch:
    """The one launch whose name holds `part`."""
    hits = [f for f in found if part in f.name]
    assert len(hits) == 1, (part, found)
    return hits[0]
