// Runs the launch rules of one source of the loss operators (SOURCE) on the
// host, with stand-ins for the HIP runtime's entry points that count launches
// and start none: every row length within the operators' range gets a kernel
// that takes it, and a kernel is refused for rows that it does not take.
#include SOURCE

#include <cstdlib>

static int launches = 0;

extern "C" {
hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) {
    launches++;
    return hipSuccess;
}
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
    *grid = *block = dim3(1);
    *lds = 0;
    *s = nullptr;
    return hipSuccess;
}
void** __hipRegisterFatBinary(const void*) {
    static void* handle;
    return &handle;
}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
void __hipUnregisterFatBinary(void**) {}
}

namespace ga {
ga_status fail(ga_status code, const char*, ...) { return code; }
ga_status check_launch(const char*) { return GA_OK; }
}  // namespace ga

using namespace ga;

static void expect(bool taken, ga_status s, const char* what, long long n) {
    if ((s == GA_OK) == taken && launches == (taken ? 1 : 0)) {
        launches = 0;
        return;
    }
    std::printf("%s: a row of %lld: status %d, %d launches\n", what, n, s, launches);
    std::exit(1);
}

// Row lengths: all up to 20000, then ever larger steps and both sides of the
// powers of two times a vector.
template <class F> static void lengths(F f) {
    for (int64_t v = 1; v < 20000; v++) f(v);
    for (int64_t v = 20000; v < INT32_MAX; v += 1 + v / 1500) f(v);
    for (int64_t b = 1 << 14; b < INT32_MAX; b *= 2)
        for (int64_t v = b - 9; v <= b + 9; v++) f(v);
    for (int64_t v = 16384; v < 200000; v += 1024)
        for (int64_t d = -8; d <= 8; d++) f(v + d);
    f(INT32_MAX);
}

#if defined(TOP)
template <ga_dtype DT> static void run() {
    TopArgs a = {};
    for (int i = 1; i <= GA_MAX_WORKERS; i++) a.rows.start[i] = 5;
    constexpr int E = RowVec<DT>::kElems;
    lengths([&](int64_t v) {
        for (int k : {1, 16, 384, 385, 1024}) {
            a.V = v;
            a.K = k;
            expect(true, launch_rows<DT>(a, nullptr), "top", v);
        }
    });
    auto v = [&](int64_t n) -> TopArgs& {
        a.V = n;
        return a;
    };
    for (int64_t less = 1; less <= 3 * E; less += E - 1) {
        expect(false, launch_top<DT, 512, 2, false>(v(1024 * E - less), nullptr), "top in rounds", a.V);
        expect(false, launch_top<DT, 1024, 2, false>(v(2048 * E - less), nullptr), "top in rounds", a.V);
        expect(false, launch_top<DT, 256, 2, true>(v(512 * E + less), nullptr), "top held", a.V);
    }
    expect(true, launch_top<DT, 512, 2, false>(v(1024 * E), nullptr), "top in rounds", a.V);
    expect(true, launch_top<DT, 256, 2, true>(v(512 * E), nullptr), "top held", a.V);
}
#elif defined(DISTILL)
template <ga_dtype DT> static void run() {
    DistillArgs a = {};
    a.K = 4;
    const ga::Launch l = {dim3(1), 0, nullptr};
    constexpr int E = RowVec<DT>::kElems;
    lengths([&](int64_t v) {
        a.V = v;
        expect(true, launch_rows<DT>(a, true, l), "distill", v);
        expect(true, launch_rows<DT>(a, false, l), "distill, the loss alone", v);
    });
    auto held = [&](bool taken, int64_t n) {
        a.V = n;
        expect(taken, launch<DT, 512, true, 10, true>(a, l), "distill held", n);
    };
    held(false, 5120 * E - 1);
    held(true, 5120 * E);
    held(true, 6144 * E + E - 1);
    held(false, 6145 * E);
}
#else
template <ga_dtype DT> static void run() {
    BalanceArgs a = {};
    for (int score : {0, 1})
        for (int E = 1; E <= GA_MAX_EXPERTS; E++) {
            a.E = E;
            ga::Launch l = {};
            l.units.n = 3;
            l.score = (ga_score)score;
            expect(true, launch_rows(a, DT, team_for(E, DT), l), "balance", E);
            l.alone = true;
            expect(true, launch_rows(a, DT, team_of(E, 1), l), "balance alone", E);
        }
    const ga::Launch l = {};
    a.E = 65;
    expect(false, launch_team<DT, 1, 64, 1>(a, l), "balance by single elements", a.E);
    expect(false, launch_team<DT, 4, 64, 4>(a, l), "balance by fours", a.E);
    a.E = 68;
    expect(false, launch_team<DT, 4, 16, 1>(a, l), "balance by fours", a.E);
}
#endif

int main() {
    run<GA_F32>();
    run<GA_BF16>();
    std::puts("ok");
}
