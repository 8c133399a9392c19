"""Child process of the launch-grid tests: makes operator calls on stand-in
addresses with tests/c/launch_record.c in the place of the HIP launch, and
prints what each would have launched.

    python tests/launch_grid_child.py RECORD.so < calls.json

calls: [[call, {argument: value}], ...] as in test_operators_abi_cpu.call_*, where
an argument is a number or [constructor, {field: value}]. Prints one JSON list of
[status, message, [[grid x, grid y, threads], ...]]. No GPU is visible to it."""

import ctypes
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
for name in ("HIP_VISIBLE_DEVICES", "ROCR_VISIBLE_DEVICES", "CUDA_VISIBLE_DEVICES"):
    os.environ[name] = ""
record = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)      # before libqknorm.so: found first
record.launch_record_at.restype = ctypes.POINTER(ctypes.c_uint)

import test_operators_abi_cpu as calls  # noqa: E402

BUILD = {"operand": calls.operand, "grad": calls.grad, "rope": calls.rope, "cache": calls.cache, "batch": calls.batch}

out = []
for name, kw in json.load(sys.stdin):
    args = {k: BUILD[v[0]](**v[1]) if isinstance(v, list) else v for k, v in kw.items()}
    record.launch_record_clear()
    rc = getattr(calls, "call_" + name)(**args)
    n = record.launch_record_count()
    out.append([rc, calls.message(), [record.launch_record_at(i)[:3] for i in range(n)]])
print(json.dumps(out))
