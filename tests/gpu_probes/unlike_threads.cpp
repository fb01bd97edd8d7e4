// Three host threads call the expert products over 1024, 2 and 300 experts on one GPU, each with its
// own stream, buffers and workspace. A call's shared memory grows with its experts, so that a
// thread must not undo what another one's launch needs. Prints the number of calls that failed.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>

#include "ft_moe.h"

static std::atomic<int> failed{0}, ready{0};

static void work(int E)
{
    const int P = 16, N = 64, K = 128;
    cudaStream_t s;
    void *x, *w, *y, *dw, *ws, *scale;
    int *offs;
    if (cudaSetDevice(0) || cudaStreamCreate(&s) || cudaMalloc(&x, P * K * 2) || cudaMalloc(&w, (size_t)E * N * K * 2) ||
        cudaMalloc(&y, P * N * 4) || cudaMalloc(&dw, (size_t)E * N * K * 4) || cudaMalloc(&ws, 256) ||
        cudaMalloc(&scale, 4 * (E + P)) || cudaMalloc(&offs, 4 * (E + 1)) || cudaMemset(x, 0, P * K * 2) ||
        cudaMemset(w, 0, (size_t)E * N * K * 2) || cudaMemset(scale, 0, 4 * (E + P))) {
        failed = 1 << 20;
        ++ready;
        return;
    }
    std::vector<int> h(E + 1, P);  // the first expert owns all rows
    h[0] = 0;
    if (cudaMemcpy(offs, h.data(), 4 * (E + 1), cudaMemcpyHostToDevice)) failed = 1 << 20;
    ++ready;
    while (ready < 3) std::this_thread::yield();
    for (int i = 0; i < 5000; ++i) {
        const ft_status r[3] = {
            ft_moe_group_gemm(x, K, w, offs, E, P, N, K, y, N, FT_DTYPE_F32, ws, 256, s),
            ft_moe_group_gemm_wgrad(x, N, x, K, offs, E, P, N, K, dw, FT_DTYPE_F32, 0, ws, 256, s),
            ft_moe_group_gemm_fp8(x, K, (const float *)scale, P, w, (const float *)scale, offs, E, P, N, K, y, N, FT_DTYPE_F32,
                                  ws, 256, s)};
        for (ft_status one : r)
            if (one != FT_OK && failed++ < 3) std::printf("E %d, call %d: %s\n", E, i, ft_last_error());
        if (i % 256 == 255) cudaStreamSynchronize(s);
    }
    if (ft_moe_read_status(ws, s) != FT_OK) ++failed;
}

int main()
{
    std::thread a(work, 1024), b(work, 2), c(work, 300);
    a.join();
    b.join();
    c.join();
    std::printf("failed calls: %d\n", failed.load());
    return failed != 0;
}
