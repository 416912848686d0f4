// api_util.cuh -- host helpers of the C entry points (argument checks, workspace layout).
#pragma once

#include <cstdint>

#include "common.cuh"

namespace moe {
namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxDevices = 64;

size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int num_sms_current() {
    static int cache[kMaxDevices] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    if (cache[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 148;
        cache[dev] = n;
    }
    return cache[dev];
}

// The routed gate_up may cut its tiles' K steps into up to kSplitMax slices when its tiles
// cannot fill the GPU (a few tokens, or a few experts), if the slices' fp32 partial sums
// (kSplitMax planes of [T*K, 2f]) take at most 64 MiB; one ticket per tile, bounded by the
// tiles of 16-row blocks: min(E, T*K) + T*K/16 + 1 row blocks of f/128 feature blocks.
constexpr int kSplitMax = 4;
bool gate_up_split_ok(long long T, long long K, long long f) {
    return 4ll * kSplitMax * T * K * 2 * f <= (64ll << 20);
}
long long gate_up_ticket_cap(long long T, long long E, long long K, long long f) {
    if (!gate_up_split_ok(T, K, f)) return 0;
    const long long rows = T * K;
    return (std::min(E, rows) + rows / 16 + 1) * (f / 128);
}

int check_shape(int T, int D, int E, int K, int f, int fs) {
    if (T < 0 || D <= 0 || E <= 0 || K <= 0 || f <= 0 || fs < 0) return MOE_ERR_ARG;
    if (E > 512 || K > 16 || K > E) return MOE_ERR_UNSUPPORTED;
    if (D % 128 || D > 8192 || f % 128 || f > 8192 || fs % 128 || fs > 8192)
        return MOE_ERR_UNSUPPORTED;
    if (static_cast<long long>(T) * K >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

template <class P>
P* at(void* ws, size_t off) {
    return reinterpret_cast<P*>(static_cast<uint8_t*>(ws) + off);
}

}  // namespace
}  // namespace moe
