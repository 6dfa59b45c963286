// Checks of tensor arguments shared by the C-ABI files of a training step.
#pragma once

#include "disco_internal.h"

namespace disco {

// One tensor argument: what it is called, where it lies and how long it is.
struct Arg {
    const char* name;
    const void* p;
    int64_t bytes;
    int align;      // of one element
    bool required;
    int in_place = -1;   // an output: the index of the input it may be, exactly
};

// Device, alignment and overlap checks of a call: outputs may overlap nothing.
inline int check_args(const Arg* ins, int n_in, const Arg* outs, int n_out) {
    int dev = -1;
    int rc = current_device(&dev);
    if (rc != DISCO_OK) return rc;
    for (int k = 0; k < n_in + n_out; ++k) {
        const Arg& a = k < n_in ? ins[k] : outs[k - n_in];
        if (a.p == nullptr && !a.required) continue;
        if ((rc = check_device_ptr(a.p, a.name, dev)) != DISCO_OK) return rc;
        if (reinterpret_cast<uintptr_t>(a.p) % a.align != 0)
            return set_error(DISCO_EINVAL, "%s is not aligned to its element size", a.name);
    }
    for (int i = 0; i < n_out; ++i) {
        if (outs[i].p == nullptr) continue;
        for (int k = 0; k < n_in; ++k)
            if (ins[k].p && !(outs[i].in_place == k && outs[i].p == ins[k].p) &&
                overlap(outs[i].p, outs[i].bytes, ins[k].p, ins[k].bytes))
                return set_error(DISCO_EINVAL, "%s overlaps %s", outs[i].name, ins[k].name);
        for (int k = i + 1; k < n_out; ++k)
            if (outs[k].p && overlap(outs[i].p, outs[i].bytes, outs[k].p, outs[k].bytes))
                return set_error(DISCO_EINVAL, "%s overlaps %s", outs[i].name, outs[k].name);
    }
    return DISCO_OK;
}

}  // namespace disco
