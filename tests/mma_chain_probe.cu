// Measures what the f16 warp MMA drops when one accumulator takes 32 MMAs of 16 E4M3 products each, with the
// helpers of the page-selection kernel and in its one chain.  Prints, per kind of data, the largest error in
// units of (n / 4 + 32 * 5 / 4) 2^-23 S, n the number of products that are not zero and S the sum of their
// magnitudes: the error of sums whose addends (the products and, once per MMA, the running sum) are each cut
// below 2^-25 of the largest one's leading bit, and whose result is cut to the 24 bits of fp32 once per MMA.
//
// What is dropped adds up behind one large product: equal ones of one sign, just below 2^-f of its leading bit,
// in all places of every MMA, or in one, two (every pair) or four of them: two cuts per MMA would drop two
// products there.
#include <cmath>
#include <cstdio>
#include <cstdlib>
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
    float acc[4] = {};
    for (int s = 0; s < STEPS; ++s) {
        uint32_t a0, a1, a2, a3, b0, b1;
        fa8::e4m3x4_to_h2(*reinterpret_cast<const uint32_t *>(a + r * K + 16 * s + 4 * c), a0, a2);
        fa8::e4m3x4_to_h2(*reinterpret_cast<const uint32_t *>(a + (r + 8) * K + 16 * s + 4 * c), a1, a3);
        fa8::e4m3x4_to_h2(*reinterpret_cast<const uint32_t *>(b + r * K + 16 * s + 4 * c), b0, b1);
        fa8::mma_f16(acc, a0, a1, a2, a3, b0, b1);
    }
    for (int e = 0; e < 4; ++e) out[(r + 8 * (e >> 1)) * 8 + 2 * c + (e & 1)] = acc[e];
}

static double dec(uint8_t c) {
    const int e = (c >> 3) & 15, m = c & 7;
    const double v = e == 0 ? m * pow(2.0, -9) : (8 + m) * pow(2.0, e - 10);
    return c & 0x80 ? -v : v;
}
// code of m / 8 * 2^e, m from 8 to 15 (e from -6 to 8), or of m / 4 * 2^-7, m from 4 to 7 (e = -7)
static uint8_t enc(int m, int e) { return (uint8_t)(e < -6 ? m / 2 : (e + 7) << 3 | (m - 8)); }

int main() {
    const int blocks = 256;
    uint8_t *da, *db;
    float *dout;
    if (cudaMalloc(&da, blocks * 16 * K) || cudaMalloc(&db, blocks * 8 * K) || cudaMalloc(&dout, blocks * 128 * 4)) return 2;
    std::vector<uint8_t> a(blocks * 16 * K), b(blocks * 8 * K);
    auto run = [&](const char *name) {
        if (cudaMemcpy(da, a.data(), a.size(), cudaMemcpyHostToDevice) || cudaMemcpy(db, b.data(), b.size(), cudaMemcpyHostToDevice)) exit(3);
        probe<<<blocks, 32>>>(da, db, dout);
        std::vector<float> out(blocks * 128);
        if (cudaMemcpy(out.data(), dout, out.size() * 4, cudaMemcpyDeviceToHost) != cudaSuccess) exit(3);
        double worst = 0;
        for (int bl = 0; bl < blocks; ++bl)
            for (int i = 0; i < 16; ++i)
                for (int j = 0; j < 8; ++j) {
                    double s = 0, mag = 0;  // sums of E4M3 products are exact in fp64
                    int n = 0;
                    for (int k = 0; k < K; ++k) {
                        const double x = dec(a[(bl * 16 + i) * K + k]) * dec(b[(bl * 8 + j) * K + k]);
                        s += x;
                        mag += fabs(x);
                        n += x != 0;
                    }
                    if (mag > 0) worst = fmax(worst, fabs(out[bl * 128 + i * 8 + j] - s) / ((n + 5 * STEPS) * pow(2.0, -25) * mag));
                }
        printf("%s|%.6g\n", name, worst);
    };
    const char *kinds[] = {"around one", "all magnitudes", "cancelling", "one large", "positive", "positive, all magnitudes", "one large, positive ones behind"};
    for (int kind = 0; kind < 7; ++kind) {
        srand(kind + 1);
        auto code = [&](int k) -> uint8_t {
            const int u = rand();
            switch (kind) {
                case 0: return (uint8_t)((u & 0x80) | (0x28 + u % 0x20));            // 0.25 .. 4
                case 1: return (uint8_t)((u & 0x80) | u % 0x7F);                      // any finite code
                case 2: return (uint8_t)((k & 1 ? 0x80 : 0) | (0x70 + u % 8));        // +-128 .. 240, alternating
                case 3: return (uint8_t)(k == 7 ? 0x7E : (u & 0x80) | u % 0x20);      // 448 among small ones
                case 4: return (uint8_t)(0x20 + u % 0x30);
                case 5: return (uint8_t)(u % 0x7F);
                default: return (uint8_t)(k == 0 ? 0x7E : u % 0x28);
            }
        };
        for (size_t i = 0; i < a.size(); ++i) a[i] = code(i % K);
        for (size_t i = 0; i < b.size(); ++i) b[i] = code(i % K);
        run(kinds[kind]);
    }
    // block bl: the large product in place bl % 16 of the first MMA.  m = 16: row i of a has products behind it in
    // the first 2 (i + 1) MMAs only; m = 1, 2, 4: in places bl / 16, bl % 16 and two drawn ones of every MMA
    for (int m : {16, 1, 2, 4})
        for (int f = 20; f < 30; ++f)
            for (int sign = 0; sign < 2; ++sign) {
                srand(f);
                const int ea = (16 - f) / 2, eb = 16 - f - ea;  // 1.75 2^ea x 1.125 2^eb = 0.98 2^(17 - f)
                for (int bl = 0; bl < blocks; ++bl) {
                    int places = m == 16 ? 0xFFFF : 1 << bl / 16;
                    if (m == 2 || m == 4) places |= 1 << bl % 16;
                    if (m == 4) places |= 1 << rand() % 16 | 1 << rand() % 16;
                    for (int i = 0; i < 16; ++i)
                        for (int k = 0; k < K; ++k)
                            a[(bl * 16 + i) * K + k] = (m < 16 || k < 32 * (i + 1)) && (places >> k % 16 & 1) ? (uint8_t)(enc(9, ea) | (sign ? 0x80 : 0)) : 0;
                    for (int j = 0; j < 8; ++j)
                        for (int k = 0; k < K; ++k) b[(bl * 8 + j) * K + k] = enc(14, eb);
                    for (int i = 0; i < 16; ++i)
                        for (int j = 0; j < 8; ++j) a[(bl * 16 + i) * K + bl % 16] = b[(bl * 8 + j) * K + bl % 16] = 0x7E;
                }
                char name[80];
                snprintf(name, sizeof(name), "one large first, %d an MMA behind at 2^-%d of it, %s", m, f, sign ? "other sign" : "same sign");
                run(name);
            }
    return 0;
}
