/* Stands in for the CUDA runtime's launches (LD_PRELOAD; no GPU is needed).
 *
 * cudaFuncSetAttribute keeps what was last set for each kernel, as the runtime
 * does.  One call can be held: having set its value, it returns only after
 * another call for the same kernel has set another.
 * cudaLaunchKernelExC refuses a launch with more shared memory than was set,
 * as the runtime does, and counts the others. */
#define _GNU_SOURCE
#include <pthread.h>
#include <stddef.h>
#include <time.h>

enum { KERNELS = 256, DEFAULT_SMEM = 48 * 1024 };
static pthread_mutex_t lock = PTHREAD_MUTEX_INITIALIZER;
static pthread_cond_t changed = PTHREAD_COND_INITIALIZER;
static const void* kernels[KERNELS];
static int smem[KERNELS], calls[KERNELS];
static int hold, held, launches, refused;

struct dim { unsigned x, y, z; };
struct config {
    struct dim grid, block;
    size_t smem;
    void* stream;
    void* attrs;
    unsigned n;
};

static int place(const void* f) {
    int i = 0;
    while (i < KERNELS - 1 && kernels[i] && kernels[i] != f) ++i;
    kernels[i] = f;
    return i;
}

void fake_hold(void) { hold = 1; }
int fake_held(void) { return held; }
int fake_launches(void) { return launches; }
int fake_refused(void) { return refused; }

int cudaGetDevice(int* d) { return *d = 0; }
int cudaFuncSetAttribute(const void* f, int attr, int value) {
    pthread_mutex_lock(&lock);
    const int i = place(f);
    ++calls[i];
    pthread_cond_broadcast(&changed);
    if (attr == 8) smem[i] = value;              /* MaxDynamicSharedMemorySize */
    if (hold) {
        struct timespec until;
        clock_gettime(CLOCK_REALTIME, &until);
        until.tv_sec += 3;
        hold = 0;
        held = 1;
        const int seen = calls[i];
        while (calls[i] == seen && pthread_cond_timedwait(&changed, &lock, &until) == 0) {
        }
        /* the other call has returned, and its launch been made */
        pthread_mutex_unlock(&lock);
        nanosleep(&(struct timespec){0, 200000000}, NULL);
        pthread_mutex_lock(&lock);
    }
    pthread_mutex_unlock(&lock);
    return 0;
}
int cudaLaunchKernelExC(const struct config* c, const void* f, void** args) {
    (void)args;
    pthread_mutex_lock(&lock);
    const int i = place(f);
    const int limit = smem[i] > DEFAULT_SMEM ? smem[i] : DEFAULT_SMEM;
    const int bad = c->smem > (size_t)limit;
    refused += bad;
    launches += !bad;
    pthread_mutex_unlock(&lock);
    return bad;                                  /* cudaErrorInvalidValue */
}
