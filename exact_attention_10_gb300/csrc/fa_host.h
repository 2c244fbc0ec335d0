// fa_host.h -- host-side checks shared by the translation units of the C ABI
// (defined in fa_api.cu): the current device, argument ranges, pointers.
#pragma once

#include <cstddef>

#include "fa.h"

namespace fa_host {

struct DeviceInfo {
    bool probed = false;
    bool supported = false;   // compute capability 10.3
    int sms = 0;
};

// The device `dev`, probed once; null if it is out of range.
const DeviceInfo *device_info(int dev);

bool ranges_overlap(const void *a, size_t na, const void *b, size_t nb);

// Rows (tokens) of one tensor, at most: kernels index them with 32 bits, and a
// block's or cluster's stride past the last one must not wrap.
constexpr long long kMaxRows = (1ll << 31) - 65536;

// Device (or managed) memory of device `dev`.
bool is_device_pointer(const void *p, int dev);

// One argument of a call: its bytes, and whether the call writes it.
struct Arg {
    const void *p;
    size_t bytes;
    bool out;
    unsigned align;   // required alignment in bytes (a power of two)
};

// What every entry point checks of its pointers before anything is enqueued:
// none null, all aligned, no output overlapping another argument (inputs may
// alias one another), the current device supported (its number and
// properties returned) and holding all of them.
fa_status check_args(const Arg *args, int n, int *dev, const DeviceInfo **info);

// Raise a kernel's dynamic shared-memory limit on device `dev`, once: `set`
// holds one flag per device (kMaxDevices), zero at first, for this kernel.
constexpr int kMaxDevices = 64;
fa_status allow_smem(const void *kern, int smem, int dev, bool *set);

}  // namespace fa_host
