"""Stream capture through the CUDA runtime itself, so that a test can look at
the nodes of a graph, launch it, or only capture it."""
from __future__ import annotations

import ctypes

import torch

KERNEL, MEMSET = 0, 2                     # cudaGraphNodeType
_PRIORITY = 8                             # cudaLaunchAttributePriority
_rt = None


def runtime():
    global _rt
    if _rt is None:
        torch.cuda.init()
        _rt = ctypes.CDLL("libcudart.so.13")   # the process's own, by its soname
    return _rt


def _call(name, *args):
    e = getattr(runtime(), name)(*args)
    assert e == 0, f"{name}: CUDA error {e}"


class Graph:
    """What `work()` enqueues on `stream`, captured the way torch.cuda.graph
    does.  Nothing of it may allocate through PyTorch."""

    def __init__(self, stream, work):
        self.stream, self.exec = stream, None
        handle = ctypes.c_void_p(stream.cuda_stream)
        self.graph = ctypes.c_void_p()
        torch.cuda.synchronize()
        _call("cudaStreamBeginCapture", handle, 0)       # cudaStreamCaptureModeGlobal
        try:
            with torch.cuda.stream(stream):
                work()
        finally:
            _call("cudaStreamEndCapture", handle, ctypes.byref(self.graph))

    def nodes(self):
        n = ctypes.c_size_t(0)
        _call("cudaGraphGetNodes", self.graph, None, ctypes.byref(n))
        if n.value == 0:
            return []
        nodes = (ctypes.c_void_p * n.value)()
        _call("cudaGraphGetNodes", self.graph, nodes, ctypes.byref(n))
        return [ctypes.c_void_p(v) for v in nodes]

    def types(self):
        out = []
        for node in self.nodes():
            t = ctypes.c_int(-1)
            _call("cudaGraphNodeGetType", node, ctypes.byref(t))
            out.append(t.value)
        return out

    def kernel_priorities(self):
        out = []
        for node, t in zip(self.nodes(), self.types()):
            if t == KERNEL:
                value = (ctypes.c_int * 16)()            # cudaLaunchAttributeValue: 64 bytes
                _call("cudaGraphKernelNodeGetAttribute", node, _PRIORITY, value)
                out.append(value[0])
        return out

    def programmatic_edges(self):
        """How many kernels may start before the one ahead of them has ended."""
        n = ctypes.c_size_t(0)
        _call("cudaGraphGetEdges", self.graph, None, None, None, ctypes.byref(n))
        if n.value == 0:
            return 0
        ends = [(ctypes.c_void_p * n.value)() for _ in range(2)]
        data = (ctypes.c_ubyte * (8 * n.value))()        # cudaGraphEdgeData: two ports, the type, reserved
        _call("cudaGraphGetEdges", self.graph, *ends, data, ctypes.byref(n))
        return sum(data[8 * i + 2] == 1 for i in range(n.value))

    def launch(self):
        if self.exec is None:
            self.exec = ctypes.c_void_p()
            _call("cudaGraphInstantiate", ctypes.byref(self.exec), self.graph, ctypes.c_ulonglong(0))
        _call("cudaGraphLaunch", self.exec, ctypes.c_void_p(self.stream.cuda_stream))

    def close(self):
        if self.exec is not None:
            _call("cudaGraphExecDestroy", self.exec)
        _call("cudaGraphDestroy", self.graph)
