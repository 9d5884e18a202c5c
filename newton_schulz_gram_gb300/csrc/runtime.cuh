// Host-side runtime shared by the C ABI translation units: error texts, the
// per-device state with its cached workspace, launch accounting and the
// tensor-map encoder. Defined in api.cu.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <string>

#include "gns.h"
#include "ptx.cuh"

namespace gns {

// Records the text gns_last_error() returns and passes the code on.
int fail(int code, const std::string& msg);
int cuda_fail(cudaError_t e, const char* what);

#define CK(call)                                                        \
    do {                                                                \
        cudaError_t e_ = static_cast<cudaError_t>(call);                \
        if (e_ != cudaSuccess) return cuda_fail(e_, #call);             \
    } while (0)

#define RET(call)                 \
    do {                          \
        int r_ = (call);          \
        if (r_ != GNS_OK) return r_; \
    } while (0)

struct DeviceState {
    int device = -1;
    int num_sms = 0;
    int cc_major = 0, cc_minor = 0;
    char* ws = nullptr;
    size_t ws_bytes = 0;
    int* err = nullptr;      // status block: [0] status word, [1] abort mark (see DevStatus)
    int epoch = 0;           // number of the current call on this device
    DevStatus status{};      // the current call's device-side error reporting
    float* stage = nullptr;  // device staging for the host-buffer entry point
    size_t stage_bytes = 0;
    cudaStream_t h2d = nullptr, d2h = nullptr;  // copy streams of the host-buffer entry point
};

// State of the current device, created on first use.
int get_state(DeviceState** out);

// Starts a call on a device: a new epoch for its kernels' abort mark. The
// second form hands it to the caller, for calls that may run beside others.
void begin_call(DeviceState& st);
DevStatus new_call(DeviceState& st);

int ensure_workspace(DeviceState& st, size_t bytes);

// Intermediate memory of one call, in the order of its stream; one per call.
// Calls on other streams have their own, and in a stream capture it is part of
// the graph, so no later call can free or overwrite it. (The workspace above is
// one buffer per device that a larger call replaces.)
// A stream's buffer stays for its next call, which cannot begin before this one
// is done with it, and is locked from take() on, so that two threads that
// launch on one stream do not mix their kernels. Allocating for every call
// instead took the host 2 us of the 15 to 20 (48 rows through the fused layer,
// alone: 44 us, 50 with two allocations).
struct ScratchSlot;
class Scratch {
public:
    Scratch() = default;
    Scratch(const Scratch&) = delete;
    Scratch& operator=(const Scratch&) = delete;
    ~Scratch();
    int take(DeviceState& st, size_t bytes, cudaStream_t s);
    char* data() const { return p_; }

private:
    char* p_ = nullptr;
    ScratchSlot* slot_ = nullptr;  // locked; null for memory of this call alone
    cudaStream_t s_ = nullptr;
};

// Kernel classes of gns_profile_read().
enum KernelClass {
    kClsGemm = 0,
    kClsNorm = 1,
    kClsMuon = 2,
    kClsCopy = 3,
    kClsFp8Gemm = 4,
    kClsFp8Cast = 5,
    kClsMoe = 6,
    kClsDropout = 7,
    kClsLayerNorm = 8,
    kClsEmbedding = 9,
    kNumCls = 10
};

// Accounting around one launch (see gns_launch_count, gns_profile_enable).
struct LaunchMark {
    cudaEvent_t a, b;  // null unless profiling is on
    int cls;
};
LaunchMark launch_begin(int cls, cudaStream_t s);
void launch_end(const LaunchMark& m, cudaStream_t s);

template <typename F>
int counted_launch(int cls, cudaStream_t s, F&& fn) {
    const LaunchMark m = launch_begin(cls, s);
    const int r = fn();
    launch_end(m, s);
    return r;
}

#define LAUNCH(cls, call) CK(::gns::counted_launch((cls), s, [&]() { return static_cast<int>(call); }))

// The driver's tensor-map encoder (null when unavailable).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

}  // namespace gns
