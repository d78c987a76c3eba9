// k3_runtime.cu -- host state shared by every launch of the library: the device
// error word, the SM count, the dynamic shared-memory limits raised for each
// kernel, and the streams whose last weights may not be complete.
//
// The first three are kept per device (the current device at the call), since a
// CUDA context holds its own copy of each, and their first-time set-up is
// guarded so that concurrent first calls from several host threads are safe.
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>
#include <vector>

#include "k3_device.cuh"

// The device error word: one zero-initialised int in every device that loads
// the library, kept until the process exits.  No allocation is involved, so
// every entry point (the allocation-free one included) reports through it.
static __device__ int g_device_error;

namespace k3 {
namespace {
constexpr int kMaxDevices = 64;
std::once_flag g_err_once[kMaxDevices];
int *g_err_addr[kMaxDevices];
std::atomic<int> g_sms[kMaxDevices];
std::mutex g_smem_mu;
struct SmemLimit {
    int dev;
    const void *fn;
    size_t bytes;
};
std::vector<SmemLimit> g_smem;


// Streams on which a call has written what may be weights and no kernel that loads
// weights early has followed yet; the mark goes with the first one, which waits for
// everything before it.  In a capture the mark is the capture's and stays: its
// streams may depend on one another, and a graph is recorded once.  When the table
// is full every stream counts as marked, and captures up to the newest id that left
// the ring do.
std::mutex g_written_mu;
constexpr int kMaxWritten = 256, kMaxCaptures = 64;
std::atomic<int> g_n_written{0};      // marked streams; kMaxWritten + 1: all
std::atomic<int> g_n_captures{0};     // captures marked so far
uintptr_t g_written[kMaxWritten];
unsigned long long g_capture[kMaxCaptures], g_capture_floor;

// One more than the id of the capture that s takes part in, 0 for none.  (The legacy
// stream beside another's capture gives an error and takes part in none.)
unsigned long long capture_of(cudaStream_t s)
{
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(s, &st, &id) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return st == cudaStreamCaptureStatusNone ? 0 : id + 1;
}
// One key for the two names of the legacy default stream.
uintptr_t stream_key(cudaStream_t s) { return s == cudaStreamLegacy ? 0 : (uintptr_t)s; }

int current_device()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return -1;
    }
    return dev;
}
}  // namespace

// Device address of the error word on the current device (host code cannot
// use the symbol's name as an address); looked up once per device.
int *device_error_word()
{
    const int dev = current_device();
    if (dev < 0) return nullptr;
    std::call_once(g_err_once[dev], [dev] {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_error) == cudaSuccess)
            g_err_addr[dev] = (int *)p;
        else
            cudaGetLastError();
    });
    return g_err_addr[dev];
}

int num_sms()
{
    const int dev = current_device();
    if (dev < 0) return 1;
    int n = g_sms[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            n = 1;
        }
        g_sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Raises kernel fn's dynamic shared-memory limit on the current device to at
// least `bytes` (once per device and size); K3MOE_ECUDA if refused.
int ensure_smem(const void *fn, size_t bytes)
{
    if (bytes <= 48 * 1024) return K3MOE_OK;
    const int dev = current_device();
    if (dev < 0) return K3MOE_ENODEV;
    std::lock_guard<std::mutex> lock(g_smem_mu);
    for (SmemLimit &l : g_smem)
        if (l.dev == dev && l.fn == fn) {
            if (l.bytes >= bytes) return K3MOE_OK;
            if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
                cudaGetLastError();
                return K3MOE_ECUDA;
            }
            l.bytes = bytes;
            return K3MOE_OK;
        }
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    g_smem.push_back({dev, fn, bytes});
    return K3MOE_OK;
}

// The table alone, by key and capture id.
void written_note(uintptr_t stream, unsigned long long capture)
{
    std::lock_guard<std::mutex> lock(g_written_mu);
    if (capture) {
        const int n = g_n_captures.load(std::memory_order_relaxed);
        for (int i = 0; i < n && i < kMaxCaptures; i++)
            if (g_capture[i] == capture) return;
        unsigned long long &slot = g_capture[n % kMaxCaptures];
        if (n >= kMaxCaptures && slot > g_capture_floor) g_capture_floor = slot;
        slot = capture;
        g_n_captures.store(n < 2 * kMaxCaptures ? n + 1 : n + 1 - kMaxCaptures, std::memory_order_relaxed);
        return;
    }
    const int n = g_n_written.load(std::memory_order_relaxed);
    if (n > kMaxWritten) return;
    for (int i = 0; i < n; i++)
        if (g_written[i] == stream) return;
    if (n < kMaxWritten) g_written[n] = stream;
    g_n_written.store(n + 1, std::memory_order_relaxed);
}
bool written_take(uintptr_t stream, unsigned long long capture)
{
    std::lock_guard<std::mutex> lock(g_written_mu);
    if (capture) {
        const int n = g_n_captures.load(std::memory_order_relaxed);
        for (int i = 0; i < n && i < kMaxCaptures; i++)
            if (g_capture[i] == capture) return true;
        return capture <= g_capture_floor;
    }
    const int n = g_n_written.load(std::memory_order_relaxed);
    if (n > kMaxWritten) return true;
    for (int i = 0; i < n; i++)
        if (g_written[i] == stream) {
            // one handle names the per-thread default streams of all threads: kept
            if (stream != (uintptr_t)cudaStreamPerThread) {
                g_written[i] = g_written[n - 1];
                g_n_written.store(n - 1, std::memory_order_relaxed);
            }
            return true;
        }
    return false;
}

// A lock that fails counts as marked; no exception reaches an entry point.
void note_weight_writes(cudaStream_t s) noexcept
{
    try {
        written_note(stream_key(s), capture_of(s));
    } catch (...) {
        g_n_written.store(kMaxWritten + 1, std::memory_order_relaxed);
    }
}
bool weights_settled(cudaStream_t s) noexcept
{
    // nothing marked anywhere: no question to the driver
    if (g_n_written.load(std::memory_order_relaxed) == 0 && g_n_captures.load(std::memory_order_relaxed) == 0)
        return true;
    try {
        return !written_take(stream_key(s), capture_of(s));
    } catch (...) {
        return false;
    }
}

}  // namespace k3
