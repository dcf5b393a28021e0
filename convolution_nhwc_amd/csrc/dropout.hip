// Dropout with a mask drawn from a counter-based generator and never stored:
//     y = residual + (keep ? x / (1 - p) : 0)
// keep(i) compares word i % 4 of Philox4x32-10 at counter (i / 4, offset) under
// the key `seed` with p * 2^32.  Philox is the published generator of Salmon,
// Moraes, Dror and Shaw ("Parallel random numbers: as easy as 1, 2, 3", 2011):
// ten rounds of two 32 x 32 -> 64 bit products and exclusive-ors, the key
// advanced by two Weyl constants; one evaluation serves four elements, so the
// mask of any element can be drawn anywhere without state.
//
// All 32 bits of a word decide an element: with fewer, p would be rounded (16
// bits move p = 0.1 by 4e-6) for half the products.
//
// Bound by memory where large: 50176 x 384 bf16 with a residual take 19 us, 6.1
// TB/s (two reads a write, where a copy of 1 GiB has one and reaches 5.1).
#include "mix.h"

namespace cnhwc {
namespace {

constexpr uint32_t kPhiloxM0 = 0xD2511F53u, kPhiloxM1 = 0xCD9E8D57u;
constexpr uint32_t kPhiloxW0 = 0x9E3779B9u, kPhiloxW1 = 0xBB67AE85u;

struct Philox4 {
    uint32_t w[4];
};

__device__ inline Philox4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
    uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32);
    uint32_t c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
    uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = uint64_t(kPhiloxM0) * c0, p1 = uint64_t(kPhiloxM1) * c2;
        c0 = uint32_t(p1 >> 32) ^ c1 ^ k0;
        c2 = uint32_t(p0 >> 32) ^ c3 ^ k1;
        c1 = uint32_t(p1);
        c3 = uint32_t(p0);
        k0 += kPhiloxW0;
        k1 += kPhiloxW1;
    }
    return Philox4{{c0, c1, c2, c3}};
}

// Each thread takes vectors of V elements (V / 4 generator blocks).  With every
// stride dense the tensors are one run of n elements; otherwise a vector is
// cut where its row ends.
template <typename T, bool RES, bool FLAT>
__global__ __launch_bounds__(256) void dropout_kernel(const DropArgs a) {
    constexpr int V = kVec<T>, ES = kElemBytes<T>;
    const uint64_t offset = a.offset + (a.device_offset ? *a.device_offset : 0);
    const int64_t nvec = (a.n + V - 1) / V;
    const char* xp = static_cast<const char*>(a.x);
    const char* rp = static_cast<const char*>(a.residual);
    char* yp = static_cast<char*>(a.y);
    for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < nvec; v += int64_t(gridDim.x) * 256) {
        const int64_t i0 = v * V;
        int64_t xo, ro = 0, yo;
        int n = int(a.n - i0 < V ? a.n - i0 : V);
        int64_t row = 0, col = 0;
        if constexpr (FLAT) {
            xo = ro = yo = i0;
        } else {
            row = a.n <= 0xffffffffll ? int64_t(uint32_t(i0) / uint32_t(a.c)) : i0 / a.c;
            col = i0 - row * a.c;
            xo = row * a.x_stride + col;
            yo = row * a.y_stride + col;
            if (RES) ro = row * a.res_stride + col;
        }
        if (FLAT || col + n <= a.c) {
            const i32x4 xv = load_n<T>(xp + xo * ES, n);
            i32x4 rv = {0, 0, 0, 0};
            if constexpr (RES) rv = load_n<T>(rp + ro * ES, n);
            float f[V];
#pragma unroll
            for (int q = 0; q < V / 4; ++q) {
                const Philox4 w = philox(uint64_t(i0 / 4 + q), offset, a.seed);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int k = 4 * q + e;
                    const float t = w.w[e] >= a.threshold ? elem<T>(xv, k) * a.scale : 0.0f;
                    f[k] = RES ? t + elem<T>(rv, k) : t;
                }
            }
            store_n<T>(yp + yo * ES, pack_vec<T>(f), n);
        } else {
            // the vector crosses one or more row ends
            for (int q = 0; q < V / 4 && 4 * q < n; ++q) {
                const Philox4 w = philox(uint64_t(i0 / 4 + q), offset, a.seed);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (4 * q + e < n) {
                        float t = w.w[e] >= a.threshold ? load1<T>(xp + (row * a.x_stride + col) * ES) * a.scale : 0.0f;
                        if (RES) t += load1<T>(rp + (row * a.res_stride + col) * ES);
                        store1<T>(yp + (row * a.y_stride + col) * ES, t);
                        if (++col == a.c) {
                            col = 0;
                            ++row;
                        }
                    }
                }
            }
        }
    }
}

template <typename T>
void launch(const DropArgs& a, hipStream_t st) {
    const int64_t nvec = (a.n + kVec<T> - 1) / kVec<T>;
    const int64_t want = (nvec + 255) / 256;
    const dim3 grid((unsigned)(want < kNumCUs * 32 ? want : kNumCUs * 32));
    if (a.flat) {
        if (a.residual) dropout_kernel<T, true, true><<<grid, 256, 0, st>>>(a);
        else dropout_kernel<T, false, true><<<grid, 256, 0, st>>>(a);
    } else {
        if (a.residual) dropout_kernel<T, true, false><<<grid, 256, 0, st>>>(a);
        else dropout_kernel<T, false, false><<<grid, 256, 0, st>>>(a);
    }
}

}  // namespace

int launch_dropout(int dtype, const DropArgs& a, hipStream_t st) {
    if (dtype == CNHWC_F16) launch<F16>(a, st);
    else if (dtype == CNHWC_BF16) launch<BF16>(a, st);
    else launch<F32>(a, st);
    return CNHWC_OK;
}

}  // namespace cnhwc
