/* Stand-ins for the three runtime calls of wgs_check_error, preloaded ahead of
 * the CUDA runtime: the device's error words are host variables, told apart by
 * their symbols in the order of their first use.  No GPU. */
#include <stddef.h>
#include <string.h>

enum { kWords = 8 };
static const void *symbol[kWords];
static unsigned int word[kWords];

static unsigned int *find(const void *s) {
    for (int i = 0; i < kWords; ++i) {
        if (!symbol[i]) symbol[i] = s;
        if (symbol[i] == s) return word + i;
    }
    return NULL;
}

void fake_set_word(int i, unsigned int v) { word[i] = v; }

int cudaMemcpyFromSymbolAsync(void *dst, const void *s, size_t n, size_t offset, int kind, void *stream) {
    unsigned int *w = find(s);
    (void)kind, (void)stream;
    if (!w || n != sizeof(*w) || offset != 0) return 1;
    memcpy(dst, w, n);
    return 0;
}

int cudaMemcpyToSymbolAsync(const void *s, const void *src, size_t n, size_t offset, int kind, void *stream) {
    unsigned int *w = find(s);
    (void)kind, (void)stream;
    if (!w || n != sizeof(*w) || offset != 0) return 1;
    memcpy(w, src, n);
    return 0;
}

int cudaStreamSynchronize(void *stream) {
    (void)stream;
    return 0;
}
