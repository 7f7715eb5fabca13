// The runs in which the scan's kernels load rows of states (Run of sq_scan_device.h), built for the host
// under AddressSanitizer: every lane of a row, for every number of states that the kernels take, with the
// row a heap block of exactly its size, and in a block whose elements behind the row are NaN.  A run
// holds the row's elements, and 0 for those past its end.
#include <hip/hip_runtime.h>

#undef __device__
#define __device__ __host__ __attribute__((device))
#define __uint_as_float(x) __builtin_bit_cast(float, (uint32_t)(x))
#include "sq_scan_device.h"

#include <cstdio>
#include <memory>

using namespace sqimpl;

namespace {
long g_mismatches = 0, g_runs = 0;

void put(float *p, float v) { *p = v; }
void put(Bf16 *p, float v) { p->bits = (uint16_t)(__builtin_bit_cast(uint32_t, v) >> 16); }

template <typename XT, int NL, bool FITS>
void lanes(const char *kernel, int count) {
    for (int behind : {0, 64}) {
        const std::unique_ptr<XT[]> row(new XT[count + behind]);
        for (int i = 0; i < count + behind; ++i) put(&row[i], i < count ? 1.0f + i : __builtin_nanf(""));
        for (int lane = 0; lane < 4; ++lane) {
            Run<XT, NL, FITS> run;
            run.load(row.get(), lane * NL, count);
            run.end(lane * NL, count);
            ++g_runs;
            for (int i = 0; i < NL; ++i) {
                const int at = lane * NL + i;
                const float want = at < count ? 1.0f + at : 0.0f;
                if (!(run[i] == want) && ++g_mismatches <= 20)
                    std::printf("MISMATCH %s, %d states of %d bytes, %d behind: element %d is %g\n", kernel, count, (int)sizeof(XT), behind, at, run[i]);
            }
        }
    }
}

template <typename XT>
void kernels() {
    // sq_prompt.hip: sixteens of states, a quarter of them a lane
    lanes<XT, 4, false>("prompt", 8), lanes<XT, 4, false>("prompt", 16);
    lanes<XT, 8, false>("prompt", 24), lanes<XT, 8, false>("prompt", 32);
    lanes<XT, 12, false>("prompt", 40), lanes<XT, 12, false>("prompt", 48);
    lanes<XT, 16, false>("prompt", 56), lanes<XT, 16, false>("prompt", 64);
    // sq_scan.hip: up to 32 states a quarter of them a lane
    lanes<XT, 2, true>("scan", 8), lanes<XT, 4, true>("scan", 16), lanes<XT, 6, true>("scan", 24), lanes<XT, 8, true>("scan", 32);
    lanes<XT, 12, false>("scan", 40), lanes<XT, 12, false>("scan", 48);
    lanes<XT, 16, false>("scan", 56), lanes<XT, 16, false>("scan", 64);
}
}  // namespace

int main() {
    kernels<Bf16>();
    kernels<float>();
    std::printf("%ld runs, %ld mismatches\n", g_runs, g_mismatches);
    std::puts(g_mismatches ? "FAILED" : "ALL OK");
    return g_mismatches != 0;
}
