"""What the block norms' backward pass enqueues, seen without a GPU: a child
process loads tests/c/launch_recorder.c in front of libecho, makes the calls
with made-up pointers (nothing is launched, so nothing is read) and prints
the recorded launches."""
import ctypes
import json
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = 1 << 20          # 16-byte aligned, never dereferenced


def build(folder):
    lib = os.path.join(str(folder), "liblaunch_recorder.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", lib, os.path.join(HERE, "c", "launch_recorder.c"), "-ldl"],
                   check=True)
    return lib


def backward_launches(lib, calls):
    """For each dict of a call (T, H, gate_tokens, gate, dw): its status and [kernel's name, grid, block] of each launch."""
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib, json.dumps(calls)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return json.loads(r.stdout.splitlines()[-1])


def _backward(echo, T, H, gate_tokens=0, gate=False, dw=True):
    a = echo.NormArgs()
    a.T, a.H, a.gate_tokens = T, H, gate_tokens
    a.ld_x = a.ld_r = a.ld_gate = H
    a.x_dtype = a.r_dtype = a.w_dtype = echo.BF16
    a.post, a.eps, a.res_scale, a.block_scale = 1, 1e-5, 1.0, 1.0
    a.x = a.r = FAKE
    g = echo.NormGrads()
    g.ld_dh = g.ld_dr_out = g.ld_dx = g.ld_dr = g.ld_dgate = H
    g.dh_dtype = echo.BF16
    g.dh = g.dr_out = g.dx = g.dr = FAKE
    if gate:
        a.gate = g.dgate = FAKE
    if dw:
        g.dw_post = g.dw_pre = FAKE
    g.workspace, g.workspace_bytes = FAKE, echo.echo_block_norm_backward_workspace_bytes(T, H)
    return echo.lib().echo_block_norm_backward(ctypes.byref(a), ctypes.byref(g), None)


def _main(lib, calls):
    rec = ctypes.CDLL(lib, mode=ctypes.RTLD_GLOBAL)
    rec.recorder_name.restype = ctypes.c_char_p
    sys.path.insert(0, os.path.dirname(HERE))
    from error_feedback_quant_amd import echo
    out = []
    for c in json.loads(calls):
        rec.recorder_clear()
        rc = _backward(echo, **c)
        got = []
        for i in range(rec.recorder_count()):
            dims = (ctypes.c_uint32 * 6)()
            rec.recorder_dims(i, dims)
            got.append([rec.recorder_name(i).decode(), list(dims[:3]), list(dims[3:])])
        out.append([rc, got])
    print(json.dumps(out))


if __name__ == "__main__":
    _main(*sys.argv[1:])
