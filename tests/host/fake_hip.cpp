// A stand-in for the part of the HIP runtime that libw8a16.so calls, for tests
// of its host code on machines without a GPU: loaded before the library with
// global symbols, so that the library binds to it.  Memory is malloc's,
// launches run nothing and are recorded.
//
// fake_no_memory: C++ allocations of the calling thread fail while it is set.
// fake_pause_us: sleep after each launch, so that other threads get between
// one call's launches where nothing keeps them out.
#include <chrono>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <new>
#include <thread>
#include <vector>

namespace {

struct Dim {
    uint32_t x, y, z;
};
struct Launch {
    uint64_t thread, stream, blocks, threads;
};
struct Config {
    Dim grid, block;
    size_t shared;
    void *stream;
};

constexpr int kInvalidConfiguration = 9;
std::mutex g_mutex;
std::vector<Launch> g_launches;
uint64_t g_pause_us = 0;
thread_local std::vector<Config> g_configs;
thread_local int g_error = 0;
thread_local uint64_t g_thread = 0;
thread_local bool g_no_memory = false;
uint8_t g_symbol[32];

}  // namespace

void *operator new(size_t n)
{
    void *p = g_no_memory ? nullptr : std::malloc(n ? n : 1);
    if (!p)
        throw std::bad_alloc();
    return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, size_t) noexcept { std::free(p); }

extern "C" {

void fake_no_memory(int on) { g_no_memory = on != 0; }
void fake_pause_us(uint64_t us) { g_pause_us = us; }
void fake_thread(uint64_t id) { g_thread = id; }
uint64_t fake_launches() { return g_launches.size(); }
void fake_launch(uint64_t i, uint64_t *out)
{
    const Launch &l = g_launches[i];
    out[0] = l.thread, out[1] = l.stream, out[2] = l.blocks, out[3] = l.threads;
}
void fake_forget() { g_launches.clear(); }

void **__hipRegisterFatBinary(const void *)
{
    static void *handle;
    return &handle;
}
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *, char *, const char *, unsigned, void *, void *, void *, void *,
                           int *)
{
}
void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}

int __hipPushCallConfiguration(Dim grid, Dim block, size_t shared, void *stream)
{
    g_configs.push_back({grid, block, shared, stream});
    return 0;
}
int __hipPopCallConfiguration(Dim *grid, Dim *block, size_t *shared, void **stream)
{
    const Config c = g_configs.back();
    g_configs.pop_back();
    *grid = c.grid, *block = c.block, *shared = c.shared, *stream = c.stream;
    return 0;
}
int hipLaunchKernel(const void *, Dim grid, Dim block, void **, size_t, void *stream)
{
    const uint64_t blocks = (uint64_t)grid.x * grid.y * grid.z, threads = (uint64_t)block.x * block.y * block.z;
    if (!blocks || !threads || blocks * threads >= 1ull << 32)
        return g_error = kInvalidConfiguration;
    {
        const std::lock_guard<std::mutex> lock(g_mutex);
        g_launches.push_back({g_thread, (uint64_t)(uintptr_t)stream, blocks, threads});
    }
    if (g_pause_us)
        std::this_thread::sleep_for(std::chrono::microseconds(g_pause_us));
    return 0;
}
int hipGetLastError()
{
    const int e = g_error;
    g_error = 0;
    return e;
}
const char *hipGetErrorString(int) { return "refused by the stand-in"; }
int hipGetDevice(int *dev)
{
    *dev = 0;
    return 0;
}
int hipDeviceGetAttribute(int *value, int, int)
{
    *value = 256;
    return 0;
}
int hipMalloc(void **p, size_t) { return (*p = std::malloc(16)) ? 0 : 2; }      // (never touched)
int hipFree(void *p)
{
    std::free(p);
    return 0;
}
int hipMemsetAsync(void *, int, size_t, void *) { return 0; }
int hipFuncSetAttribute(const void *, int, int) { return 0; }
int hipGetSymbolAddress(void **p, const void *)
{
    *p = g_symbol;
    return 0;
}
int hipStreamIsCapturing(void *, int *status)
{
    *status = 0;
    return 0;
}
int hipStreamSynchronize(void *) { return 0; }

}  // extern "C"
