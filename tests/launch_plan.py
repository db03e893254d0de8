"""What libdg.so launches for given calls, without a GPU:

    python launch_plan.py RECORDER LIBRARY < calls.json > plan.json

A call is [entry point, argument, ...]; "p" stands for a device pointer (never
followed), null for none, "w" for a workspace and the next argument, its size.
Prints the names of all kernels in the library and, per call, its status and
those it launched.  Run in a process of its own: RECORDER takes the place of the
HIP runtime there."""
import ctypes
import json
import sys


def main(recorder, library):
    rec = ctypes.CDLL(recorder, mode=ctypes.RTLD_GLOBAL)
    rec.recorded_kernel.restype = rec.recorded_launch.restype = ctypes.c_char_p
    lib = ctypes.CDLL(library)
    plans = []
    for name, *args in json.load(sys.stdin):
        fn = getattr(lib, name)
        before = rec.recorded_launches()
        status = fn(*[ctypes.c_void_p(0x10000) if a in ("p", "w") else ctypes.c_void_p(0) if a is None
                      else ctypes.c_int64(a) for a in args])
        plans.append([status, [rec.recorded_launch(i).decode()
                               for i in range(before, rec.recorded_launches())]])
    print(json.dumps({"kernels": [rec.recorded_kernel(i).decode() for i in range(rec.recorded_kernels())],
                      "plans": plans}))


if __name__ == "__main__":
    main(*sys.argv[1:3])
