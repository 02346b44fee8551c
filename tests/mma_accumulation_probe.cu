// Measures how far the f16 warp MMA's fp32 accumulation of E4M3 products is from the exact sum, with the
// helpers of the page-selection kernel: chains of 16-product MMAs over K = 512 products, two
// accumulators, as the kernel runs them.  Prints, per kind of data, the largest error in units of
// 2^-23 times the number of MMAs times sum |a_k| * max |b|.
#include <cstdio>
#include <cstdlib>
#include <cmath>
#include <vector>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa8_kernel.cuh"
#include "fa8_pages.cuh"

constexpr int K = 512, STEPS = K / 16;

// a (16 x K) and b (8 x K), E4M3; out (16 x 8).  The contraction order is free, so lane (r, c) takes the
// k elements 4 c .. 4 c + 3 of each 16.
__global__ void probe(const uint8_t *a, const uint8_t *b, float *out) {
    a += blockIdx.x * 16 * K;
    b += blockIdx.x * 8 * K;
    out += blockIdx.x * 128;
    const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
    float acc[2][4] = {};
    for (int s = 0; s < STEPS; ++s) {
        uint32_t a0, a1, a2, a3, b0, b1;
        fa8::e4m3x4_to_h2(*reinterpret_cast<const uint32_t *>(a + r * K + 16 * s + 4 * c), a0, a2);
        fa8::e4m3x4_to_h2(*reinterpret_cast<const uint32_t *>(a + (r + 8) * K + 16 * s + 4 * c), a1, a3);
        fa8::e4m3x4_to_h2(*reinterpret_cast<const uint32_t *>(b + r * K + 16 * s + 4 * c), b0, b1);
        if (s & 1) fa8::mma_f16(acc[1], a0, a1, a2, a3, b0, b1);
        else fa8::mma_f16(acc[0], a0, a1, a2, a3, b0, b1);
    }
    for (int e = 0; e < 4; ++e) out[(r + 8 * (e >> 1)) * 8 + 2 * c + (e & 1)] = acc[0][e] + acc[1][e];
}

static double dec(uint8_t c) {
    const int e = (c >> 3) & 15, m = c & 7;
    const double v = e == 0 ? m * pow(2.0, -9) : (8 + m) * pow(2.0, e - 10);
    return c & 0x80 ? -v : v;
}

int main() {
    const char *kinds[] = {"around one", "all magnitudes", "cancelling", "one large", "positive"};
    const int blocks = 256;
    uint8_t *da, *db;
    float *dout;
    if (cudaMalloc(&da, blocks * 16 * K) || cudaMalloc(&db, blocks * 8 * K) || cudaMalloc(&dout, blocks * 128 * 4)) return 2;
    for (int kind = 0; kind < 5; ++kind) {
        std::vector<uint8_t> a(blocks * 16 * K), b(blocks * 8 * K);
        srand(kind + 1);
        auto code = [&](int k) -> uint8_t {
            const int u = rand();
            switch (kind) {
                case 0: return (uint8_t)((u & 0x80) | (0x28 + u % 0x20));            // 0.25 .. 4
                case 1: return (uint8_t)((u & 0x80) | u % 0x7F);                      // any finite code
                case 2: return (uint8_t)((k & 1 ? 0x80 : 0) | (0x70 + u % 8));        // +-128 .. 240, alternating
                case 3: return (uint8_t)(k == 7 ? 0x7E : (u & 0x80) | u % 0x20);      // 448 among small ones
                default: return (uint8_t)(0x20 + u % 0x30);
            }
        };
        for (size_t i = 0; i < a.size(); ++i) a[i] = code(i % K);
        for (size_t i = 0; i < b.size(); ++i) b[i] = code(i % K);
        cudaMemcpy(da, a.data(), a.size(), cudaMemcpyHostToDevice);
        cudaMemcpy(db, b.data(), b.size(), cudaMemcpyHostToDevice);
        probe<<<blocks, 32>>>(da, db, dout);
        std::vector<float> out(blocks * 128);
        if (cudaMemcpy(out.data(), dout, out.size() * 4, cudaMemcpyDeviceToHost) != cudaSuccess) return 3;
        double worst = 0;
        for (int bl = 0; bl < blocks; ++bl)
            for (int i = 0; i < 16; ++i)
                for (int j = 0; j < 8; ++j) {
                    double s = 0, l1 = 0, mx = 0;  // sums of E4M3 products are exact in fp64
                    for (int k = 0; k < K; ++k) {
                        const double x = dec(a[(bl * 16 + i) * K + k]), y = dec(b[(bl * 8 + j) * K + k]);
                        s += x * y;
                        l1 += fabs(y);
                        mx = fmax(mx, fabs(x));
                    }
                    worst = fmax(worst, fabs(out[bl * 128 + i * 8 + j] - s) / (STEPS * pow(2.0, -23) * l1 * mx));
                }
        printf("%s|%.6g\n", kinds[kind], worst);
    }
    return 0;
}
